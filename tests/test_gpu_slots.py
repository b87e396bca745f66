"""GPU: copies between the pools' slots, bit for bit against indexing."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def expected(pool, source, target):
    new = pool.clone()
    for s, t in zip(source, target):
        if 0 <= t < pool.shape[0] and s < pool.shape[0]:
            new[t] = pool[s] if s >= 0 else 0
    return new


def pool_of(shape, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if dtype.is_floating_point:
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)
    return torch.randint(-100, 100, shape, generator=gen, device="cuda").to(dtype)


PAIRS = [([0], [1]), ([2, 1], [1, 2]), ([3, 3, 3, -1], [0, 1, 2, 4]), ([1, 2, 3, 4, 0], [0, 1, 2, 3, 4]), ([4], [4]),
         ([5, 0, 1], [0, 1, 2]), ([0, 1], [-1, 9]), ([-1], [3]), ([-7, 2], [0, -3])]


@pytest.mark.parametrize("source,target", PAIRS, ids=str)
@pytest.mark.parametrize("shape,dtype", [((5, 3, 7, 9), torch.float32), ((5, 11, 3), torch.bfloat16), ((5, 33), torch.int8),
                                         ((5, 1), torch.bfloat16), ((5, 2, 64, 128), torch.float32)], ids=str)
def test_one_pool(source, target, shape, dtype):
    pool = pool_of(shape, dtype, 1)
    want = expected(pool, source, target)
    cc.state_copy(pool, ints(source), ints(target))
    assert torch.equal(pool, want)


@pytest.mark.parametrize("n", [1, 7, 64, 128, 129, 600, 1024, 1025, 8192])
def test_permutations(n):
    """Every slot is a source and a target: a rotation and a shuffle of all, which a copy in place would tear."""
    gen = torch.Generator().manual_seed(n)
    pools = [pool_of((n, 5, 31), torch.float32, n), pool_of((n, 3, 2), torch.bfloat16, n + 1)]
    order = torch.randperm(n, generator=gen)
    for source in (order, torch.arange(n).roll(1)):
        want = [p[source.cuda()] for p in pools]
        cc.state_copy(pools, source.int().cuda(), torch.arange(n, dtype=torch.int32, device="cuda"))
        assert all(torch.equal(p, w) for p, w in zip(pools, want))


def test_strided_slots_keep_what_is_between():
    wide = torch.randn(6, 100, device="cuda")
    inside = wide[:, 3:3 + 60].view(6, 5, 12)
    conv = torch.randn(6, 3, 40, device="cuda").bfloat16().transpose(1, 2)  # [slots, channels, 3], channels contiguous
    before, conv_before = wide.clone(), conv.clone()
    source, target = [4, 0, -1], [0, 4, 2]
    cc.state_copy([inside, conv], ints(source), ints(target))
    assert torch.equal(inside, expected(before[:, 3:63].reshape(6, 5, 12), source, target))
    assert torch.equal(conv, expected(conv_before, source, target))
    assert torch.equal(wide[:, :3], before[:, :3]) and torch.equal(wide[:, 63:], before[:, 63:])


def test_unaligned_bytes():
    flat = torch.randint(0, 255, (4 * 37 + 3,), dtype=torch.uint8, device="cuda")
    before = flat.clone()
    pool = flat[3:].view(4, 37)
    want = expected(before[3:].view(4, 37), [1, 0], [0, 3])
    cc.state_copy(pool, ints([1, 0]), ints([0, 3]))
    assert torch.equal(pool, want) and torch.equal(flat[:3], before[:3])


def test_pools_of_other_sizes():
    """A pair outside one pool's slots leaves that pool and moves the others; pools without slots or bytes are nothing."""
    a, b = torch.randn(4, 6, device="cuda"), torch.randn(8, 6, device="cuda")
    wa, wb = expected(a, [6, 1], [0, 2]), expected(b, [6, 1], [0, 2])
    cc.state_copy([a, torch.empty(0, 3, device="cuda"), b, torch.empty(8, 0, device="cuda")], ints([6, 1]), ints([0, 2]))
    assert torch.equal(a, wa) and torch.equal(b, wb)
    cc.state_copy([a, b], ints([]), ints([]))
    assert torch.equal(a, wa)


def test_infinities_and_nan_are_bits():
    pool = torch.full((3, 20), float("nan"), device="cuda")
    pool[1] = float("inf")
    pool[2] = -0.0
    bits = pool.view(torch.int32).clone()
    cc.state_copy(pool, ints([1, 2, 0]), ints([0, 1, 2]))
    assert torch.equal(pool.view(torch.int32), bits[[1, 2, 0]])
    cc.state_copy(pool, ints([-1]), ints([2]))
    assert (pool.view(torch.int32)[2] == 0).all()


def test_offsets_past_32_bits():
    pool = torch.empty(3, 1 << 30, dtype=torch.int16, device="cuda")
    view = pool[:, -1000:]
    view.copy_(pool_of((3, 1000), torch.int16, 3))
    want = expected(view.clone(), [0, 2], [2, 0])
    cc.state_copy(view, ints([0, 2]), ints([2, 0]))
    assert torch.equal(view, want)


def test_fork_then_decode_in_a_graph():
    """A prompt's states forked to two more slots and one cleared, then one token each: captured and replayed."""
    H, P, N = 2, 16, 32
    pool, conv = torch.randn(5, H, P, N, device="cuda"), torch.randn(5, 64, 3, device="cuda").bfloat16()
    start, conv_start = pool.clone(), conv.clone()
    source, target = ints([0, 0, -1]), ints([1, 2, 3])
    ci = ints([0, 1, 2, 3])
    q, k = (torch.randn(4, 1, N, device="cuda").bfloat16() for _ in range(2))
    v, dt = torch.randn(4, H, P, device="cuda").bfloat16(), torch.randn(4, H, device="cuda")
    A = -torch.ones(H, device="cuda")

    def work():
        cc.state_copy([conv, pool], source, target)
        return cc.delta_state_update(q, k, v, dt, dt, A, state_pool=pool, cache_indices=ci)

    def again():
        pool.copy_(start)
        conv.copy_(conv_start)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for _ in range(3):
        v.mul_(-1.25)
        again()
        graph.replay()
        torch.cuda.synchronize()
        got = captured.clone(), pool.clone(), conv.clone()
        again()
        want = work(), pool, conv
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(conv[1], conv_start[0]) and (conv[3] == 0).all()
