"""Failures of different kinds are recorded beside each other: none hides or erases another.  The wait that runs out is
the injected one of the chunk step (one copy and its barrier arrival are skipped); the bad index is a slot beyond
the pool, which the kernel does not follow."""

import pytest

torch = pytest.importorskip("torch")

from tests.parity import seeded

pytestmark = pytest.mark.gpu


@pytest.fixture
def fail(lib):
    """Calls that record a run-out wait ("wait") and an index out of range ("index")."""
    from chunked_prefill_attention_gb300 import q8attn as Q
    assert Q.device_status(clear=True)[0] == Q.Q8A_OK
    q = seeded((1, 128, 1, 64), 1, "cuda", torch.float16)
    planes = [Q.q8kv_quantize(seeded((1, 128, 1, 64), s, "cuda")) for s in (2, 3)]
    st = Q.State(1, 1, 128, "cuda")
    pages = torch.zeros((2, 1, 1, 16, 68), dtype=torch.uint8, device="cuda")
    k = torch.zeros((1, 1, 64), device="cuda")
    beyond = torch.tensor([16], device="cuda")

    def run(kind):
        if kind == "wait":
            Q.set_wait_timeout_ns(50_000_000)
            Q.test_inject(1)
            try:
                Q.attn_chunk_step(q, *planes, 0, 128, st)
            finally:
                Q.test_inject(0)
                Q.set_wait_timeout_ns(2_000_000_000)
        else:
            Q.q8kv_append_paged(k, k, pages[0], pages[1], beyond)
        torch.cuda.synchronize()

    yield run
    Q.device_status(clear=True)
    assert Q.status() == Q.Q8A_OK and (pages == 0).all()


@pytest.mark.parametrize("order", [("wait", "index"), ("index", "wait"), ("index", "wait", "index")])
def test_a_wait_and_an_index(lib, fail, order):
    from chunked_prefill_attention_gb300 import q8attn as Q
    for kind in order:
        fail(kind)
    assert Q.status() == Q.Q8A_ERR_TIMEOUT
    role = int(lib.q8a_last_error().decode().split("role ")[1].split(")")[0])
    assert role in (1, 2, 3, 4, 5)
    for clear in (False, True):   # reading does not clear
        rc, word = Q.device_status(clear=clear)
        assert rc == Q.Q8A_ERR_TIMEOUT and word & 3 == 3 and (word >> 8) & 0xFF in (1, 2, 3, 4, 5)
    assert Q.device_status(clear=True) == (Q.Q8A_OK, 0) and Q.status() == Q.Q8A_OK


def test_each_alone(lib, fail):
    from chunked_prefill_attention_gb300 import q8attn as Q
    for kind, rc, bits in (("index", Q.Q8A_ERR_INVALID_ARG, 2), ("wait", Q.Q8A_ERR_TIMEOUT, 1)):
        fail(kind)
        assert Q.status() == rc
        got, word = Q.device_status(clear=True)
        assert got == rc and word & 3 == bits
        assert Q.device_status(clear=True) == (Q.Q8A_OK, 0)
