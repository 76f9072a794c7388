"""q8kv_extend_paged where the free pages do not suffice: they are dealt in order, and no sequence overtakes another."""

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_paged import Q, clean_status   # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

PAGE = 16


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("filler", [0, 300, 3000])   # sequences before them that need no page: one block's scan, and several rounds of it
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("padding", [0, 6000])       # one block, and many
def test_no_sequence_overtakes_one_that_waits_for_pages(Q, filler, in_place, padding):
    """A prompt that lacks more pages than are left stops every later sequence that lacks any; what needs none goes on."""
    many, few, none = (200, 0), (1, 32), (1, 5)      # new tokens, keys before: 13 pages, one page, none
    for order, served in (((many, few, none, few), (0, 0, 1, 0)), ((few, many, none, few), (1, 0, 1, 0)),
                          ((few, none, few, many), (1, 1, 1, 0)), ((few, few, few, none), (1, 1, 1, 1))):
        rows = ((1, 3),) * filler + order
        B, total = len(rows), sum(n for n, _ in rows) + padding
        new, kv = i32(*(n for n, _ in rows)), i32(*(k for _, k in rows))
        table = torch.zeros((B, 20), dtype=torch.int32, device="cuda")
        table[:, :2] = torch.arange(2 * B, device="cuda").view(B, 2) + 100
        before, free, n_free = table.clone(), torch.arange(8, dtype=torch.int32, device="cuda"), i32(8)
        out = None
        if in_place:
            out = kv, torch.empty_like(torch.cat([new, new[:1]])), *(torch.empty(total, dtype=torch.int64, device="cuda") for _ in range(2)), n_free
        lens, cu, slots, pos, left = Q.q8kv_extend_paged(new, kv, table, free, n_free, PAGE, total, out=out)
        granted = [1] * filler + list(served)
        assert lens.tolist() == [k + n * g for (n, k), g in zip(rows, granted)]
        taken = 0
        slots, pos = slots.tolist(), pos.tolist()
        for b, ((n, k), g) in enumerate(zip(rows, granted)):
            r = int(cu[b])
            assert int(cu[b + 1]) == r + n
            if not g:
                assert slots[r:r + n] == [-1] * n and pos[r:r + n] == [0] * n and torch.equal(table[b], before[b])
                continue
            at = int(table[b, k // PAGE])
            if k % PAGE == 0:
                taken += 1
                assert at == 8 - taken               # the stack's next one
            assert slots[r] == at * PAGE + k % PAGE and pos[r] == k
        assert left.tolist() == [8 - taken] and free.tolist() == list(range(8))
        assert (Q.device_status(clear=True)[0] == Q.Q8A_ERR_INVALID_ARG) == (0 in served)
