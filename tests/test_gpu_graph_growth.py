"""A captured call keeps the workspace memory that its graph holds addresses of, whatever
later calls need."""
import pytest
import torch

from streaming_sinkhorn_solver_gb300 import binding as fs
from streaming_sinkhorn_solver_gb300.workloads import random_cloud
from tests.gpu_util import to_dev
from tests.test_gpu_attention import BF, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    fs.load_library()


def attention(n, m, d=72):
    c, how, dout = make(2, n, m, 4, 2, d, BF, drop=0.1, nb=16, far=50, seed=61)

    def call():
        a = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
        return [*a, *fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **how)]
    return call


def tokens(n, m):
    c, how, _ = make(1, n, m, 8, 2, 64, BF, seed=62)
    return lambda: list(fs.fs_cross_attention(c["q"], c["k"], c["v"], **how))


def solve(n, m):
    t = to_dev(random_cloud(n, m, 3, seed=63))
    return lambda: list(fs.fs_sinkhorn_solve(t["X"], t["a"], t["Y"], t["b"], 0.1, 4))


@pytest.mark.parametrize("kind,small,large", [(attention, (150, 300), (3000, 4000)),
                                              (tokens, (2, 9000), (4, 200000)),
                                              (solve, (400, 300), (60000, 50000))])
def test_replay_after_a_larger_call(kind, small, large):
    torch.cuda.synchronize()
    fs.fs_release()
    torch.cuda.empty_cache()
    call = kind(*small)
    want = [x.clone() for x in call()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    big = kind(*large)
    for _ in range(2):
        big()
        torch.cuda.synchronize()
        # takes whatever the growth gave back, and would see a write to it
        torch.cuda.empty_cache()
        guard = [torch.full((2 ** 20,), -1, dtype=torch.int8, device="cuda") for _ in range(64)]
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert torch.equal(x, y)
        for x in guard:
            assert bool((x == -1).all())
        del guard
    graph.reset()
    fs.fs_check()


def test_release_frees_what_was_kept():
    """Heads of 65 are copied to the workspace: 70 MB and 105 MB of it."""
    call, big = attention(20000, 20000, 65), attention(30000, 30000, 65)
    torch.cuda.synchronize()
    fs.fs_release()
    torch.cuda.empty_cache()
    free, reserved = torch.cuda.mem_get_info()[0], torch.cuda.memory_reserved()

    def held():          # by the library
        torch.cuda.synchronize()
        return free - torch.cuda.mem_get_info()[0] - (torch.cuda.memory_reserved() - reserved)

    call()
    first = held()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    big()
    assert held() > 2 * first > 2 ** 27
    graph.reset()
    fs.fs_release()
    assert held() < 2 ** 25
