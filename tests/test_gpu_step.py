"""The gradient norm, AdamW and packed AdamW on the GPU against the float64
oracle (and its float32 form, bit for bit, where every operation is rounded):
types, sizes around the tiles and blocks, odd alignments, many tensors,
special values, in place and beside, plans, graphs and streams."""

import math

import numpy as np
import pytest

from gpu_util import require_gpu
from oracle import step as oracle
from step_util import adamw_bound, f32, f64, norm_bound, on_device, rounded, torch_dtype

pytestmark = pytest.mark.gpu

SIZES = [1, 3, 4, 255, 256, 257, 2047, 2049, 4095, 4097, 8192, 8193, 30011]


@pytest.fixture(scope="module")
def ar():
    require_gpu()
    import ring_allreduce_reduction_virtual_amd as ar

    return ar


def _torch():
    import torch

    return torch


# --------------------------------------------------------------------------
# gradient norm
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_norm_over_sizes(ar, dtype, offset):
    rng = np.random.default_rng(3)
    for n in SIZES + [100003]:
        g = on_device(rng.standard_normal(n).astype(np.float32), dtype, offset)
        want = oracle.grad_norm([f64(g)])
        got = f64(ar.ar_grad_norm([g]))[0]
        assert abs(got - want) <= norm_bound(want), n
        plan = ar.ar_grad_norm_init([g])
        assert f64(plan.start())[0] == got, n


@pytest.mark.parametrize("count", [1, 5, 159, 160, 161, 400])
def test_norm_over_many_tensors(ar, count):
    rng = np.random.default_rng(count)
    gs = [on_device(rng.standard_normal(int(rng.integers(0, 3000))).astype(np.float32), "bf16", i % 3)
          for i in range(count)]
    want = oracle.grad_norm([f64(g) for g in gs])
    got = f64(ar.ar_grad_norm(gs))[0]
    assert abs(got - want) <= norm_bound(want)
    plan = ar.ar_grad_norm_init(gs)
    assert abs(f64(plan.start())[0] - want) <= norm_bound(want)
    assert plan.num_launches in (1, 2)


def test_norm_of_extreme_values(ar):
    torch = _torch()
    dev = "cuda"
    assert f64(ar.ar_grad_norm([torch.empty(0, device=dev)]))[0] == 0.0
    assert f64(ar.ar_grad_norm([torch.zeros(5000, device=dev)]))[0] == 0.0
    for value in (1e30, 1e-30, 1e-42, 3e38):
        g = torch.full((20001,), value, device=dev)
        want = oracle.grad_norm([f64(g)])
        got = f64(ar.ar_grad_norm([g]))[0]
        assert got == math.inf if want > 3.5e38 else abs(got - want) <= norm_bound(want)
    for bad in (math.inf, -math.inf):
        g = torch.ones(20001, device=dev)
        g[20000] = bad
        assert f64(ar.ar_grad_norm([g, torch.ones(3, device=dev)]))[0] == math.inf
    g = torch.ones(20001, device=dev)
    g[7] = math.nan
    assert math.isnan(f64(ar.ar_grad_norm([g]))[0])


def test_norm_is_the_same_bits_every_time(ar):
    torch = _torch()
    g = torch.randn(3_000_001, device="cuda")
    first = ar.ar_grad_norm([g]).clone()
    for _ in range(5):
        assert torch.equal(ar.ar_grad_norm([g]), first)


def test_norm_past_32_bit_offsets(ar):
    """2^32 + 5 elements: each index past 32 bits counts, and only once."""
    torch = _torch()
    n = (1 << 32) + 5
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-5:] = 2.0
    g[0] = 1.0
    g[1 << 31] = 4.0
    assert f64(ar.ar_grad_norm([g]))[0] == np.float32(math.sqrt(20 + 1 + 16))
    plan = ar.ar_grad_norm_init([g])
    assert f64(plan.start())[0] == np.float32(math.sqrt(37))


# --------------------------------------------------------------------------
# AdamW, float32 states
# --------------------------------------------------------------------------

HYPER = dict(step=7, lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
TYPES = [("f32", "f32", None), ("f32", "bf16", "bf16"), ("f32", "f16", "f16"), ("f32", "f32", "bf16"),
         ("bf16", "bf16", None), ("bf16", "f32", None), ("f16", "f16", None), ("f16", "f32", None),
         ("bf16", "f16", None), ("f16", "bf16", None)]


def make_inputs(rng, n, param, grad, offset=0):
    size = 10.0 ** rng.uniform(-4, 0, n)
    p = on_device(rng.standard_normal(n).astype(np.float32), param, offset)
    g = on_device((rng.standard_normal(n) * size).astype(np.float32), grad, offset)
    m = (rng.standard_normal(n) * size * 0.3).astype(np.float32)
    v = (rng.uniform(0.5, 1.5, n) * size ** 2).astype(np.float32)
    v[rng.uniform(size=n) < 0.05] = 0.0
    return p, g, m, v


def check_param(got, p, g, m, v, dtype, factor=1.0, hyper=HYPER):
    """Parameters against float64, within the step's bound and one rounding to their type."""
    p, g, m, v = f64(p), f64(g), np.asarray(m, np.float64), np.asarray(v, np.float64)
    want, _, _ = oracle.adamw(p, g, m, v, factor=factor, **hyper)
    bound = adamw_bound(p, g, m, v, factor=factor, **{k: hyper[k] for k in ("step", "lr", "betas", "eps")})
    off = np.abs(f64(got) - want)
    assert (off <= bound + rounded(np.abs(want) + bound, dtype)).all(), float((off - bound).max())


@pytest.mark.parametrize("param,grad,copy", TYPES)
def test_adamw_types_sizes_and_alignments(ar, param, grad, copy):
    torch = _torch()
    rng = np.random.default_rng(11)
    ps, gs, ms, vs, m0, v0 = [], [], [], [], [], []
    for k, n in enumerate(SIZES):
        p, g, m, v = make_inputs(rng, n, param, grad, offset=k % 4)
        ps.append(p), gs.append(g), m0.append(m), v0.append(v)
        ms.append(on_device(m, "f32", (k + 1) % 4)), vs.append(on_device(v, "f32", (k + 2) % 4))
    norm = ar.ar_grad_norm(gs)
    factor = oracle.factor_f32(f32(norm)[0], 1.0, 0.5)
    p0 = [p.clone() for p in ps]
    copies = None if copy is None else [torch.zeros(n + 1, dtype=torch_dtype(copy), device="cuda")[1:] for n in SIZES]
    out = ([torch.full_like(p, math.nan) for p in ps], [torch.full_like(m, math.nan) for m in ms],
           [torch.full_like(v, math.nan) for v in vs])
    ar.ar_adamw(ps, gs, ms, vs, out=out, copies=copies, grad_norm=norm, max_norm=1.0, grad_scale=0.5, **HYPER)
    for k, n in enumerate(SIZES):
        want_m, want_v = oracle.moments_f32(f32(gs[k]), m0[k], v0[k], HYPER["betas"], factor)
        assert np.array_equal(f32(out[1][k]), want_m) and np.array_equal(f32(out[2][k]), want_v), n
        check_param(out[0][k], p0[k], gs[k], m0[k], v0[k], param, factor)
        assert torch.equal(ps[k], p0[k]) and np.array_equal(f32(ms[k]), m0[k]), "inputs stay"
        if copies is not None:
            assert torch.equal(copies[k], out[0][k].to(copies[k].dtype)), n
    # in place, and as a plan: the same bits
    plan = ar.ar_adamw_init(ps, gs, ms, vs, copies=copies)
    assert plan.num_launches == 1
    plan.start(grad_norm=norm, max_norm=1.0, grad_scale=0.5, **HYPER)
    for got, want in zip((ps, ms, vs), out):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_adamw_writes_nothing_beside_its_tensors(ar):
    """The elements around every tensor keep their values, whatever its length and offset."""
    torch = _torch()
    for n in (1, 5, 257, 4099):
        for offset in (0, 1, 2):
            whole = [torch.full((n + 16,), 7.0, device="cuda") for _ in range(4)]
            p, g, m, v = (w[offset:offset + n] for w in whole)
            ar.ar_adamw([p], [g], [m], [v], step=1, lr=0.1)
            for w in (whole[0], whole[2], whole[3]):
                assert (w[:offset] == 7).all() and (w[offset + n:] == 7).all()
                assert (w[offset:offset + n] != 7).all()


@pytest.mark.parametrize("count", [0, 47, 48, 49, 200])
def test_adamw_over_many_tensors(ar, count):
    """Across the lines of one launch's table; empty tensors among them."""
    torch = _torch()
    sizes = [int(x) for x in np.random.default_rng(count).integers(0, 5000, max(count, 1))]
    if count == 0:
        sizes = [0]
    ps, gs, ms, vs = ([torch.randn(n, device="cuda") for n in sizes] for _ in range(4))
    vs = [v.square() for v in vs]
    flat = [torch.cat(x) for x in (ps, gs, ms, vs)]
    planned = [[t.clone() for t in x] for x in (ps, gs, ms, vs)]
    ar.ar_adamw(ps, gs, ms, vs, **HYPER)
    if flat[0].numel():
        ar.ar_adamw([flat[0]], [flat[1]], [flat[2]], [flat[3]], **HYPER)
    for got, want in zip((ps, ms, vs), (flat[0], flat[2], flat[3])):
        assert torch.equal(torch.cat(got), want)
    plan = ar.ar_adamw_init(*planned)
    plan.start(**HYPER)
    for got, want in zip((planned[0], planned[2], planned[3]), (ps, ms, vs)):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_adamw_follows_many_steps(ar):
    """Twenty steps in place against float64, each within its own bound of the state it starts from."""
    rng = np.random.default_rng(4)
    p, g, m, v = make_inputs(rng, 5000, "f32", "f32")
    m, v = on_device(m * 0, "f32"), on_device(v * 0, "f32")
    for t in range(1, 21):
        g.copy_(_torch().from_numpy(rng.standard_normal(5000).astype(np.float32)))
        before = [x.clone() for x in (p, g, m, v)]
        hyper = dict(HYPER, step=t)
        ar.ar_adamw([p], [g], [m], [v], **hyper)
        check_param(p, before[0], before[1], f64(before[2]), f64(before[3]), "f32", hyper=hyper)


def test_adamw_nonfinite_gradients(ar):
    """They reach the elements they belong to; with skip_nonfinite nothing changes."""
    torch = _torch()
    for packed in (False, True):
        for out in (False, True):
            n = 5000
            p, g = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
            g[4321] = math.inf
            if packed:
                m, v = (ar.PackedState.zeros(n, "cuda") for _ in range(2))
                m.codes.random_(0, 256), v.codes.random_(0, 256), m.scales.fill_(120), v.scales.fill_(110)
                new = [[torch.zeros_like(p)], [ar.PackedState.zeros(n, "cuda")], [ar.PackedState.zeros(n, "cuda")]]
                call, more = ar.ar_adamw_packed, {"seed": 1}
                flat = lambda x: list(x)                                # noqa: E731
            else:
                m, v = torch.randn(n, device="cuda"), torch.rand(n, device="cuda")
                new = [[torch.zeros_like(t)] for t in (p, m, v)]
                call, more = ar.ar_adamw, {}
                flat = lambda x: [x]                                    # noqa: E731
            before = [t.clone() for t in [p] + flat(m) + flat(v)]
            norm = ar.ar_grad_norm([g])
            call([p], [g], [m], [v], out=new if out else None, grad_norm=norm, skip_nonfinite=True, **more, **HYPER)
            got = [new[0][0]] + flat(new[1][0]) + flat(new[2][0]) if out else [p] + flat(m) + flat(v)
            assert all(torch.equal(a, b) for a, b in zip(got, before))
            call([p], [g], [m], [v], **more, **HYPER)
            block = slice(4321 // 256 * 256, 4321 // 256 * 256 + 256) if packed else slice(4321, 4322)
            values = [ar.ar_unpack_states([s], k)[0] for s, k in ((m, "exp_avg"), (v, "exp_avg_sq"))] if packed \
                else [m, v]
            for t in values:
                bad = ~torch.isfinite(t)
                assert bad[block].all() and int(bad.sum()) == block.stop - block.start
            assert int((~torch.isfinite(p)).sum()) <= 1


def test_adamw_zero_states_and_eps(ar):
    """No gradient and zero states: parameters only decay; eps = 0 makes 0 / 0 of them."""
    torch = _torch()
    p = torch.ones(300, device="cuda")
    z = [torch.zeros(300, device="cuda") for _ in range(3)]
    ar.ar_adamw([p], [z[0]], [z[1]], [z[2]], step=1, lr=0.5, weight_decay=0.5)
    assert (p == 0.75).all()
    ar.ar_adamw([p], [z[0]], [z[1]], [z[2]], step=1, lr=0.5, eps=0.0)
    assert torch.isnan(p).all()


def test_adamw_past_32_bit_offsets(ar):
    """2^32 + 261 elements, float32 and packed states: the last ones are the last ones."""
    torch = _torch()
    n = (1 << 32) + 261
    p, g = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m, v = (torch.zeros(n, device="cuda") for _ in range(2))
    g[-300:] = 1.0
    g[5] = 1.0
    ar.ar_adamw([p], [g], [m], [v], step=1, lr=0.5)
    for t, want in ((p, -0.5), (m, np.float32(1 - 0.9)), (v, np.float32(1 - 0.999))):
        assert (t[-300:].float() == float(want)).all() and t[5].item() == float(want)
        assert int((t[:1000] != 0).sum()) == 1 and int((t[-1300:] != 0).sum()) == 300
    del m, v
    torch.cuda.empty_cache()
    p.zero_()
    m, v = (ar.PackedState.zeros(n, "cuda") for _ in range(2))
    plan = ar.ar_adamw_packed_init([p], [g], [m], [v])
    plan.start(step=1, lr=0.5, seed=0)
    assert (p[-300:].float() == -0.5).all() and int((p[-1300:] != 0).sum()) == 300
    assert (m.codes[-300:] != 0).all() and int((m.codes[-1300:] != 0).sum()) == 300
    # 300 = 5 of the last block, the 256 before them, 39 of the third
    assert [s > 1 for s in m.scales[-4:].tolist()] == [False, True, True, True]


# --------------------------------------------------------------------------
# packed states
# --------------------------------------------------------------------------

def packed_inputs(ar, rng, n, offset):
    """States with random codes and scales, at odd addresses."""
    def state(lo, hi, kind):
        codes = rng.integers(0, 256, n).astype(np.uint8)
        scales = rng.integers(lo, hi, oracle.blocks_of(n)).astype(np.uint8)
        return ar.PackedState(on_device(codes, "u8", offset), on_device(scales, "u8", offset + 1)), \
            oracle.unpack(codes, scales, kind).astype(np.float32)

    return state(110, 125, "exp_avg"), state(95, 120, "exp_avg_sq")


@pytest.mark.parametrize("param,grad,copy", TYPES)
def test_packed_types_sizes_and_alignments(ar, param, grad, copy):
    torch = _torch()
    rng = np.random.default_rng(12)
    sizes = [n for n in SIZES if n < 9000]
    seed, want, args = 99, [], ([], [], [], [])
    for k, n in enumerate(sizes):
        p, g, _, _ = make_inputs(rng, n, param, grad, offset=k % 4)
        (m, m32), (v, v32) = packed_inputs(ar, rng, n, k % 5)
        for a, x in zip(args, (p, g, m, v)):
            a.append(x)
        want.append((p.clone(), m32, v32))
    norm = ar.ar_grad_norm(args[1])
    factor = oracle.factor_f32(f32(norm)[0], 1.0)
    copies = None if copy is None else [torch.zeros(n, dtype=torch_dtype(copy), device="cuda") for n in sizes]

    def like(s):
        return ar.PackedState(torch.full_like(s.codes, 77), torch.full_like(s.scales, 77))

    out = ([torch.full_like(p, math.nan) for p in args[0]], [like(s) for s in args[2]], [like(s) for s in args[3]])
    ar.ar_adamw_packed(*args, out=out, copies=copies, seed=seed, grad_norm=norm, max_norm=1.0, **HYPER)
    for k, n in enumerate(sizes):
        p0, m32, v32 = want[k]
        m, v = oracle.moments_f32(f32(args[1][k]), m32, v32, HYPER["betas"], factor)
        bits = oracle.random_bits(seed, k, n)
        for got, x, kind in ((out[1][k], m, "exp_avg"), (out[2][k], v, "exp_avg_sq")):
            codes, scales = oracle.pack(x, bits, kind)
            assert np.array_equal(got.scales.cpu().numpy(), scales), (n, kind)
            assert np.array_equal(got.codes.cpu().numpy(), codes), (n, kind)
        check_param(out[0][k], p0, args[1][k], m32, v32, param, factor)
        if copies is not None:
            assert torch.equal(copies[k], out[0][k].to(copies[k].dtype))
    plan = ar.ar_adamw_packed_init(*args, copies=copies)
    assert plan.num_launches == 1
    plan.start(seed=seed, grad_norm=norm, max_norm=1.0, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(args[0], out[0]))
    for got, new in ((args[2], out[1]), (args[3], out[2])):
        assert all(torch.equal(x, y) for a, b in zip(got, new) for x, y in zip(a, b))


@pytest.mark.parametrize("count", [29, 30, 31, 32, 33, 100])
def test_packed_over_many_tensors(ar, count):
    """One call over all, a plan over all: the same bits; each tensor draws its own random bits."""
    torch = _torch()
    sizes = [int(x) for x in np.random.default_rng(count).integers(0, 3000, count)]
    args = []
    for _ in range(2):
        torch.manual_seed(count)
        ps, gs = ([torch.randn(n, device="cuda") for n in sizes] for _ in range(2))
        ms, vs = ([ar.PackedState.zeros(n, "cuda") for n in sizes] for _ in range(2))
        args.append((ps, gs, ms, vs))
    plan = ar.ar_adamw_packed_init(*args[1])
    for t in (1, 2, 3):
        ar.ar_adamw_packed(*args[0], step=t, lr=0.1, seed=t)
        plan.start(step=t, lr=0.1, seed=t)
    for a, b in zip(args[0], args[1]):
        for x, y in zip(a, b):
            for s, t in zip(x if isinstance(x, tuple) else (x,), y if isinstance(y, tuple) else (y,)):
                assert torch.equal(s, t)
    for k in (0, count - 1):
        one = [[torch.zeros_like(args[0][0][k])], [args[0][1][k]]] + \
            [[ar.PackedState.zeros(sizes[k], "cuda")] for _ in range(2)]
        ar.ar_adamw_packed(*one, step=1, lr=0.1, seed=1)
        m = oracle.moments_f32(f32(args[0][1][k]), np.zeros(sizes[k], np.float32), np.zeros(sizes[k], np.float32),
                               (0.9, 0.999), 1.0)[0]
        codes, _ = oracle.pack(m, oracle.random_bits(1, 0, sizes[k]), "exp_avg")
        assert np.array_equal(one[2][0].codes.cpu().numpy(), codes)


def test_packed_second_moment_follows_the_float32_one(ar):
    """Noisy gradients of one variance for 3,000 steps: the packed second moment's mean is the float32 one's.

    Each step's rounding is unbiased; its noise per element is at most an
    eighth of the value times sqrt(p), p = 0.1 % of it / (1/16) = 1/60 a step,
    over 500 steps of memory: 0.125 * sqrt(500 / 60) = 0.36 of the value, and
    over 65,536 elements 0.0014 of the mean.  The bound is 2 %; rounding to
    the nearest would have stopped below a tenth.
    """
    torch = _torch()
    n = 1 << 16
    gen = torch.Generator(device="cuda").manual_seed(0)
    p = [torch.zeros(n, device="cuda") for _ in range(2)]
    g = torch.zeros(n, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    pm, pv = (ar.PackedState.zeros(n, "cuda") for _ in range(2))
    plain = ar.ar_adamw_init([p[0]], [g], [m], [v])
    packed = ar.ar_adamw_packed_init([p[1]], [g], [pm], [pv])
    for t in range(1, 3001):
        g.normal_(generator=gen)
        plain.start(step=t, lr=1e-3)
        packed.start(step=t, lr=1e-3, seed=t)
    got = f64(ar.ar_unpack_states([pv], "exp_avg_sq")[0]).mean()
    assert abs(got / f64(v).mean() - 1) < 0.02
    # and the parameters walk as far
    assert 0.9 < f64(p[1]).std() / f64(p[0]).std() < 1.1


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["exp_avg", "exp_avg_sq"])
def test_unpack_every_code_and_scale(ar, dtype, kind):
    """All 256 codes at every scale byte, 0 and 255 among them."""
    codes = np.tile(np.arange(256, dtype=np.uint8), 256)
    scales = np.arange(256).astype(np.uint8)
    state = ar.PackedState(on_device(codes, "u8", 3), on_device(scales, "u8", 1))
    got = f64(ar.ar_unpack_states([state], kind, dtype=torch_dtype(dtype))[0])
    want = oracle.unpack(codes, scales, kind)
    finite = np.isfinite(want)
    assert np.array_equal(np.isnan(got), ~finite)
    with np.errstate(all="ignore"):
        # through float32 (a subnormal's rounding), then the type's own
        want = want[finite].astype(np.float32)
        exact = _torch().from_numpy(want).to(torch_dtype(dtype)).double().numpy()
    assert np.array_equal(got[finite], exact)


def test_unpack_many_and_odd(ar):
    torch = _torch()
    rng = np.random.default_rng(8)
    sizes = [1, 7, 8, 9, 255, 256, 257, 2048, 2049, 5000] * 12
    states, want = [], []
    for n in sizes:
        codes, scales = rng.integers(0, 256, n).astype(np.uint8), rng.integers(100, 140, oracle.blocks_of(n)).astype(np.uint8)
        states.append(ar.PackedState(on_device(codes, "u8", n % 7), on_device(scales, "u8", n % 3)))
        want.append(oracle.unpack(codes, scales, "exp_avg"))
    outs = [torch.full((n + 2,), 9.0, device="cuda") for n in sizes]
    ar.ar_unpack_states(states, "exp_avg", outs=[o[1:-1] for o in outs])
    for o, w in zip(outs, want):
        assert np.array_equal(f64(o[1:-1]), w) and o[0] == 9 and o[-1] == 9


# --------------------------------------------------------------------------
# plans, graphs, streams
# --------------------------------------------------------------------------

def test_step_captured_into_a_graph(ar):
    """Norm, step and unpacking captured, replayed between eager work: each replay equals the eager call."""
    torch = _torch()
    sizes = [4099, 17, 100_000]
    gs = [torch.randn(n, device="cuda") for n in sizes]
    sets = []
    for _ in range(2):
        torch.manual_seed(3)
        ps = [torch.randn(n, device="cuda") for n in sizes]
        ms, vs = ([ar.PackedState.zeros(n, "cuda") for n in sizes] for _ in range(2))
        sets.append((ps, gs, ms, vs))
    norm_plan = ar.ar_grad_norm_init(gs)
    plans = [ar.ar_adamw_packed_init(*s) for s in sets]
    config = dict(step=1, lr=0.1, seed=5, grad_norm=norm_plan.norm, max_norm=0.5)
    values = [torch.empty(n, device="cuda") for n in sizes]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        norm_plan.start()
        plans[0].start(**config)
        ar.ar_unpack_states(sets[0][2], "exp_avg", outs=values)
    for _ in range(4):
        for g in gs:
            g.normal_()
        graph.replay()
        torch.cuda.synchronize()
        ar.ar_grad_norm(gs, norm=norm_plan.norm)
        plans[1].start(**config)
        want = ar.ar_unpack_states(sets[1][2], "exp_avg")
        assert all(torch.equal(a, b) for a, b in zip(sets[0][0], sets[1][0]))
        assert all(torch.equal(a, b) for a, b in zip(values, want))


def test_plans_cannot_be_made_under_capture(ar):
    torch = _torch()
    p, g, m, v = (torch.zeros(100, device="cuda") for _ in range(4))
    need = ar.ar_update_workspace_bytes("adamw", [100])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        g.add_(1)
        with pytest.raises(ar.ArError, match="captured"):
            ar.ar_adamw_init([p], [g], [m], [v], workspace=ws)


def test_step_on_another_stream(ar):
    """Work enqueued on a stream of the caller's own, outputs made there, waited for before they are read."""
    torch = _torch()
    stream = torch.cuda.Stream()
    gs = [torch.randn(n, device="cuda") for n in (1_000_003, 5)]
    ps, ms, vs = ([torch.zeros_like(g) for g in gs] for _ in range(3))
    stream.wait_stream(torch.cuda.current_stream())
    norm = ar.ar_grad_norm(gs, stream=stream)
    ar.ar_adamw(ps, gs, ms, vs, step=1, lr=0.1, grad_norm=norm, max_norm=1.0, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    want = oracle.grad_norm([f64(g) for g in gs])
    assert abs(f64(norm)[0] - want) <= norm_bound(want)
    factor = oracle.factor_f32(f32(norm)[0], 1.0)
    zero = np.zeros(5, np.float32)
    assert np.array_equal(f32(ms[1]), oracle.moments_f32(f32(gs[1]), zero, zero, (0.9, 0.999), factor)[0])
    with pytest.raises(ValueError, match="raw handle"):
        ar.ar_grad_norm(gs, stream=stream.cuda_stream)
    ws = torch.empty(ar.ar_update_workspace_bytes("grad_norm", [g.numel() for g in gs]), dtype=torch.uint8, device="cuda")
    out = torch.zeros(1, device="cuda")
    stream.wait_stream(torch.cuda.current_stream())
    ar.ar_grad_norm(gs, norm=out, workspace=ws, stream=stream.cuda_stream)
    stream.synchronize()
    assert torch.equal(out, norm)


def test_plans_refuse_what_kernels_cannot_reach(ar):
    torch = _torch()
    import ctypes

    from ring_allreduce_reduction_virtual_amd import _lib

    L = _lib.lib()
    host = torch.zeros(64).pin_memory()
    dev = torch.zeros(64, device="cuda")
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    handle = ctypes.c_void_p()

    def init(g, count, w=None):
        ptrs, counts = (ctypes.c_void_p * 1)(g), (ctypes.c_size_t * 1)(count)
        return L.ar_grad_norm_init(ptrs, counts, 1, 0, dev.data_ptr(), ws.data_ptr() if w is None else w,
                                   ws.numel(), None, ctypes.byref(handle))

    big = torch.zeros(64, device="cuda")
    assert init(host.data_ptr(), 64) == 1 and b"host memory" in L.ar_get_last_error_detail()
    assert init(big.data_ptr(), 1 << 40) == 1
    assert init(big.data_ptr(), 64) == 0
    assert L.ar_update_free(handle) == 0


def test_binding_refusals(ar):
    torch = _torch()
    f = lambda n=8, **k: torch.zeros(n, device="cuda", **k)             # noqa: E731
    good = dict(step=1, lr=0.1)
    with pytest.raises(ValueError):
        ar.ar_grad_norm([])
    with pytest.raises(ValueError):
        ar.ar_grad_norm([torch.zeros(4)])
    with pytest.raises(TypeError):
        ar.ar_grad_norm([f(dtype=torch.float64)])
    with pytest.raises(TypeError):
        ar.ar_grad_norm([f(), f(dtype=torch.bfloat16)])
    with pytest.raises(ValueError, match="contiguous"):
        ar.ar_grad_norm([f(16)[::2]])
    with pytest.raises(ValueError, match="norm"):
        ar.ar_grad_norm([f()], norm=f(2))
    with pytest.raises(ar.ArError, match="workspace"):
        ar.ar_grad_norm([f()], workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ar.ar_adamw([f()], [f(9)], [f()], [f()], **good)
    with pytest.raises(ValueError):
        ar.ar_adamw([f()], [f()], [f(), f()], [f()], **good)
    with pytest.raises(TypeError):
        ar.ar_adamw([f()], [f()], [f(dtype=torch.bfloat16)], [f()], **good)
    with pytest.raises(TypeError, match="copies"):
        ar.ar_adamw([f(dtype=torch.bfloat16)], [f()], [f()], [f()], copies=[f(dtype=torch.bfloat16)], **good)
    x = f()
    with pytest.raises(ar.ArError, match="overlaps"):
        ar.ar_adamw([x], [x], [f()], [f()], **good)
    with pytest.raises(ar.ArError, match="overlaps"):
        ar.ar_adamw([f()], [f()], [x], [x], **good)
    y = f(16)
    with pytest.raises(ar.ArError, match="overlaps"):
        ar.ar_adamw([y[:8]], [f()], [f()], [f()], out=([y[4:12]], [f()], [f()]), **good)
    for bad in (dict(step=0), dict(lr=-1.0), dict(lr=math.nan), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)),
                dict(eps=-1.0), dict(weight_decay=math.inf), dict(grad_scale=0.0), dict(max_norm=-1.0),
                dict(max_norm=1.0), dict(skip_nonfinite=True)):
        with pytest.raises((ar.ArError, ValueError)):
            ar.ar_adamw([f()], [f()], [f()], [f()], **dict(good, **bad))
    state = ar.PackedState.zeros(8, "cuda")
    with pytest.raises(ValueError, match="PackedState"):
        ar.ar_adamw_packed([f()], [f()], [f()], [f()], seed=0, **good)
    with pytest.raises(ValueError):
        ar.ar_adamw_packed([f(300)], [f(300)], [state], [state], seed=0, **good)
    plan = ar.ar_grad_norm_init([f()])
    with pytest.raises(ValueError):
        ar.ar_adamw_start(plan, **good)
    with pytest.raises(TypeError):
        plan.start(step=1)
    plan.close()
    with pytest.raises(ValueError, match="closed"):
        plan.start()
    step = ar.ar_adamw_init([f()], [f()], [f()], [f()])
    with pytest.raises(TypeError, match="seed"):
        step.start(seed=1, **good)
    with pytest.raises(ValueError):
        ar.ar_grad_norm_start(step)


@pytest.mark.parametrize("eps", [0.0, 1e-20, 1e-13, 1e-8])
def test_packed_tiny_gradients(ar, eps):
    """Second moments down to float32's subnormals: the parameter moves as the formula says, for every eps.

    Where the hardware's root would take such a moment for 0 the step must
    not use it; the parameter is then the float32 formula's bit for bit.
    """
    torch = _torch()
    n, lr = 600, 0.25
    g = np.geomspace(1e-22, 1e-14, n).astype(np.float32)
    p = torch.zeros(n, device="cuda")
    m, v = (ar.PackedState.zeros(n, "cuda") for _ in range(2))
    ar.ar_adamw_packed([p], [torch.from_numpy(g).cuda()], [m], [v], step=1, lr=lr, eps=eps, seed=0)
    zero = np.zeros(n, np.float32)
    m32, v32 = oracle.moments_f32(g, zero, zero, (0.9, 0.999), 1.0)
    f = np.float32
    with np.errstate(all="ignore"):
        d = np.sqrt(v32) * f(1 / math.sqrt(1 - 0.999)) + f(eps)
        want = zero * f(1) - (m32 / d) * f(lr / (1 - 0.9))
    got = f32(p)
    if eps < 1e-10:
        assert np.array_equal(got, want)
    # root, its product, the sum, reciprocal, product, step size: 2 + 1 + 1 + 2 + 1 + 1 half-ulps, twice over
    assert np.allclose(got, want, rtol=16 * 2.0 ** -24, atol=1e-30)


def test_packed_blocks_of_nan_stay_with_their_own(ar):
    """A NaN block of one state keeps NaN there and in its parameters; the other state and other blocks go on."""
    torch = _torch()
    n = 1024
    p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    for bad in (0, 1):
        states = [ar.PackedState.zeros(n, "cuda") for _ in range(2)]
        states[bad].scales[2] = 255
        q = p.clone()
        ar.ar_adamw_packed([q], [g], [states[0]], [states[1]], step=1, lr=0.5, seed=3)
        block = slice(512, 768)
        assert torch.isnan(q[block]).all() and int(torch.isnan(q).sum()) == 256
        scales = [s.scales.tolist() for s in states]
        assert scales[bad][2] == 255 and 255 not in scales[bad][:2] + scales[bad][3:] + scales[1 - bad]
        other = ar.ar_unpack_states([states[1 - bad]], ("exp_avg", "exp_avg_sq")[1 - bad])[0]
        assert torch.isfinite(other).all() and (other > 0).all()


def test_packed_is_the_same_bits_every_time_and_follows_its_seed(ar):
    torch = _torch()
    g = torch.randn(100_003, device="cuda")
    got = []
    for seed in (1, 1, 2):
        p = torch.zeros_like(g)
        m, v = (ar.PackedState.zeros(g.numel(), "cuda") for _ in range(2))
        for t in (1, 2):
            ar.ar_adamw_packed([p], [g], [m], [v], step=t, lr=0.1, seed=seed)
        got.append((p, m.codes, v.codes))
    assert all(torch.equal(a, b) for a, b in zip(got[0], got[1]))
    assert (got[0][1] != got[2][1]).any() and (got[0][2] != got[2][2]).any()


@pytest.mark.parametrize("param,grad", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16")])
def test_large_forms_agree_with_small_ones(ar, param, grad):
    """A tensor in a call large enough for the other kernel form gets the bits that it gets alone."""
    torch = _torch()
    sizes = [25_000_003, 70_001, 9]
    torch.manual_seed(0)
    ps = [torch.randn(n, device="cuda").to(torch_dtype(param)) for n in sizes]
    gs = [torch.randn(n, device="cuda").to(torch_dtype(grad)) for n in sizes]
    ms, vs = ([torch.randn(n, device="cuda") for n in sizes] for _ in range(2))
    vs = [v.abs_() for v in vs]
    alone = [[t[k:k + 1] for t in ([x.clone() for x in ps], gs, [x.clone() for x in ms], [x.clone() for x in vs])]
             for k in (1, 2)]
    ar.ar_adamw(ps, gs, ms, vs, **HYPER)
    for k, a in zip((1, 2), alone):
        ar.ar_adamw(*a, **HYPER)
        assert torch.equal(a[0][0], ps[k]) and torch.equal(a[2][0], ms[k]) and torch.equal(a[3][0], vs[k])
    pm, pv = ([ar.PackedState.zeros(n, "cuda") for n in sizes] for _ in range(2))
    ar.ar_adamw_packed(ps, gs, pm, pv, seed=4, **HYPER)
    for k in (1, 2):
        want = oracle.moments_f32(f32(gs[k])[:600], np.zeros(min(600, sizes[k]), np.float32),
                                  np.zeros(min(600, sizes[k]), np.float32), HYPER["betas"], 1.0)
        for state, x, kind in ((pm[k], want[0], "exp_avg"), (pv[k], want[1], "exp_avg_sq")):
            codes, scales = oracle.pack(x, oracle.random_bits(4, k, x.size), kind)
            whole = x.size // 256 * 256 if x.size == 600 else x.size
            assert np.array_equal(state.codes.cpu().numpy()[:whole], codes[:whole])
            assert np.array_equal(state.scales.cpu().numpy()[:-(-whole // 256)], scales[:-(-whole // 256)])


@pytest.mark.parametrize("count", [34, 35, 68, 69])
def test_packed_at_the_ends_of_a_launch(ar, count):
    """As many tensors as one launch's table holds, and one more: each as if it were alone but for its number."""
    torch = _torch()
    rng = np.random.default_rng(count)
    gs = [on_device(rng.standard_normal(300 + 7 * k).astype(np.float32), "bf16", k % 3) for k in range(count)]
    ps = [torch.zeros_like(g) for g in gs]
    ms, vs = ([ar.PackedState.zeros(g.numel(), "cuda") for g in gs] for _ in range(2))
    ar.ar_adamw_packed(ps, gs, ms, vs, step=1, lr=0.1, seed=11)
    for k in (0, 33, count - 1):
        n = gs[k].numel()
        zero = np.zeros(n, np.float32)
        m, v = oracle.moments_f32(f32(gs[k]), zero, zero, (0.9, 0.999), 1.0)
        for state, x, kind in ((ms[k], m, "exp_avg"), (vs[k], v, "exp_avg_sq")):
            codes, scales = oracle.pack(x, oracle.random_bits(11, k, n), kind)
            assert np.array_equal(state.codes.cpu().numpy(), codes) and np.array_equal(state.scales.cpu().numpy(), scales)
    values = ar.ar_unpack_states(ms, "exp_avg")
    assert all(np.array_equal(f64(x), oracle.unpack(s.codes.cpu().numpy(), s.scales.cpu().numpy(), "exp_avg"))
               for x, s in zip(values, ms))


@pytest.fixture(params=["native", "python"])
def marshalling(request, monkeypatch):
    """Both ways of checking and addressing tensors."""
    from ring_allreduce_reduction_virtual_amd import step

    if request.param == "python":
        monkeypatch.setattr(step, "_fast", None)
    else:
        assert step._fast is not None, "_armarshal.so is not built"
    return request.param


def test_marshalling_both_ways(ar, marshalling):
    """Subclasses, Parameters, views, odd strides and empty tensors through every call, and the refusals' kinds."""
    torch = _torch()
    f = lambda *s, **k: torch.ones(*s, device="cuda", **k)              # noqa: E731
    whole = f(100)
    p = [torch.nn.Parameter(f(7)), whole[3:10], f(0)]
    g = (f(7), whole[50:57], f(0))                                      # a tuple will do
    m, v = ([f(7) * 0, f(7) * 0, f(0)] for _ in range(2))
    assert abs(ar.ar_grad_norm(g).item() - math.sqrt(14)) < 1e-5
    ar.ar_adamw(p, g, m, v, step=1, lr=0.5)
    assert (p[0].detach() == 0.5).all() and (whole[3:10] == 0.5).all() and (whole[10:] == 1).all()
    states = [[tuple(ar.PackedState.zeros(t.numel(), "cuda")) for t in p] for _ in range(2)]
    ar.ar_adamw_packed(p, g, *states, step=1, lr=0.5, seed=1)
    assert all(x.numel() == t.numel() for x, t in zip(ar.ar_unpack_states(states[0], "exp_avg"), p))
    x = f(4, 12)
    ys, means, _ = ar.ar_layer_norm((x[:, 1:8], f(4, 12)[:, :7]))
    assert ys[0].shape == (4, 7) and (means[0] == 1).all()
    with pytest.raises(TypeError):
        ar.ar_grad_norm([f(3), f(3, dtype=torch.bfloat16)])
    with pytest.raises(ValueError, match="contiguous"):
        ar.ar_adamw([f(6)[::2]], [f(3)], [f(3)], [f(3)], step=1, lr=0.1)
    with pytest.raises(ValueError, match="hold 3"):
        ar.ar_adamw([f(3)], [f(4)], [f(3)], [f(3)], step=1, lr=0.1)
    with pytest.raises(ValueError, match="PackedState"):
        ar.ar_unpack_states([f(3, dtype=torch.uint8)], "exp_avg")
    with pytest.raises(ValueError, match="scales"):
        ar.ar_unpack_states([(f(300, dtype=torch.uint8), f(1, dtype=torch.uint8))], "exp_avg")
    with pytest.raises(TypeError):
        ar.ar_unpack_states([(f(3), f(1, dtype=torch.uint8))], "exp_avg")
    with pytest.raises(ValueError, match="stride"):
        ar.ar_layer_norm([f(4, 8)[:, :7], f(4, 9)[:, :7]])
    with pytest.raises(ValueError, match="contiguous rows"):
        ar.ar_layer_norm([f(7, 4).t()])
    with pytest.raises(ValueError):
        ar.ar_layer_norm([f(4, 7), f(4, 8)])


@pytest.mark.parametrize("tiles", [1, 2, 3, 20, 127, 128, 129, 1024, 1500])
def test_norm_plan_started_again_and_again(ar, tiles):
    """Every start of a plan finds its workspace as the first one did, around the number of workgroups that join."""
    torch = _torch()
    tile = 8192
    g = [torch.zeros(tiles * tile // 2 - 5, device="cuda"), torch.zeros(tiles * tile - tiles * tile // 2 - 7, device="cuda")]
    plan = ar.ar_grad_norm_init(g)
    expected = []
    for k in range(1, 40):
        for t in g:
            t.fill_(float(k))
        plan.start()
        expected.append((plan.norm.clone(), k * math.sqrt(sum(t.numel() for t in g))))
    for got, want in expected:
        assert abs(f64(got)[0] - want) <= norm_bound(want)
    assert plan.num_launches == (1 if sum(-(-t.numel() // tile) for t in g) <= 128 else 2)


def test_negative_views_refused(ar):
    """A view whose elements are to be read negated holds other values in memory."""
    torch = _torch()
    g = torch._neg_view(torch.ones(64, device="cuda"))
    with pytest.raises(ValueError, match="negative"):
        ar.ar_grad_norm([g])
    x = torch._neg_view(torch.ones(2, 64, device="cuda"))
    with pytest.raises(ValueError, match="contiguous rows"):
        ar.ar_layer_norm([x])


NAN_BITS = {"f32": [0x7FC00000, 0xFFC00000, 0x7FFFFFFF, 0xFFFFFFFF, 0xFFF00001, 0xFF800001, 0xFFFF0000],
            "bf16": [0x7FC0, 0xFFC0, 0x7FFF, 0xFFFF, 0xFFF1, 0xFF81], "f16": [0x7E00, 0xFE00, 0x7FFF, 0xFFFF, 0xFF81, 0xFC01]}


@pytest.mark.parametrize("param,grad", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16")])
def test_packed_nan_gradients(ar, param, grad):
    """A NaN gradient of any sign and payload makes its block of both states NaN, and no other block."""
    torch = _torch()
    n, at = 1030, 700
    rng = np.random.default_rng(21)
    block = slice(at // 256 * 256, at // 256 * 256 + 256)
    values = rng.standard_normal(n).astype(np.float32)
    for bits in NAN_BITS[grad]:
        g = on_device(values, grad)
        whole = g.view(torch.int32 if grad == "f32" else torch.int16)
        whole[at] = bits - (1 << (32 if grad == "f32" else 16)) if bits >> (31 if grad == "f32" else 15) else bits
        assert int(torch.isnan(g).sum()) == 1
        p = torch.zeros(n, dtype=torch_dtype(param), device="cuda")
        m, v = (ar.PackedState.zeros(n, "cuda") for _ in range(2))
        ar.ar_adamw_packed([p], [g], [m], [v], step=1, lr=0.1, seed=3)
        clean = f32(g)
        clean[at] = 0.0
        zero = np.zeros(n, np.float32)
        new = oracle.moments_f32(clean, zero, zero, (0.9, 0.999), 1.0)
        for state, x, kind in ((m, new[0], "exp_avg"), (v, new[1], "exp_avg_sq")):
            codes, scales = oracle.pack(x, oracle.random_bits(3, 0, n), kind)
            codes[block], scales[at // 256] = 0, 255
            assert np.array_equal(state.scales.cpu().numpy(), scales), (hex(bits), kind)
            assert np.array_equal(state.codes.cpu().numpy(), codes), (hex(bits), kind)
            bad = torch.isnan(ar.ar_unpack_states([state], kind)[0])
            assert bad[block].all() and int(bad.sum()) == 256, (hex(bits), kind)
        assert torch.isnan(p[at]) and int((~torch.isfinite(p)).sum()) == 1, hex(bits)


@pytest.mark.parametrize("grad,copy", [("f32", None), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("eps", [1e-8, 1e-3])
def test_packed_float32_parameters_are_the_plain_steps(ar, grad, copy, eps):
    """With float32 parameters both steps round every operation: from the same states the same bits."""
    torch = _torch()
    rng = np.random.default_rng(31)
    n = 50_003
    p, g, _, _ = make_inputs(rng, n, "f32", grad)
    (m, m32), (v, v32) = packed_inputs(ar, rng, n, 1)
    config = dict(HYPER, eps=eps)
    copies = [None if copy is None else [torch.zeros(n, dtype=torch_dtype(copy), device="cuda")] for _ in range(2)]
    plain = [[p.clone()], [g], [on_device(m32, "f32")], [on_device(v32, "f32")]]
    ar.ar_adamw(*plain, copies=copies[0], **config)
    ar.ar_adamw_packed([p], [g], [m], [v], copies=copies[1], seed=2, **config)
    assert torch.equal(p, plain[0][0])
    if copy is not None:
        assert torch.equal(copies[0][0], copies[1][0])


def test_negative_norms_refused(ar):
    """The norm's own tensor neither: read in place it is another number, written it would read as minus the norm."""
    torch = _torch()
    g = [torch.ones(64, device="cuda")]
    norm = torch._neg_view(torch.full((1,), 4.0, device="cuda"))
    with pytest.raises(ValueError, match="negative"):
        ar.ar_grad_norm(g, norm=norm)
    with pytest.raises(ValueError, match="negative"):
        ar.ar_grad_norm_init(g, norm=norm)
    args = [[torch.ones(64, device="cuda")] for _ in range(4)]
    with pytest.raises(ValueError, match="negative"):
        ar.ar_adamw(*args, step=1, lr=0.1, grad_norm=norm, max_norm=1.0)
    plan = ar.ar_adamw_init(*args)
    with pytest.raises(ValueError, match="negative"):
        plan.start(step=1, lr=0.1, grad_norm=norm, max_norm=1.0)
    assert all((a[0] == 1).all() for a in args)


def versions(*tensors):
    return [t._version for t in tensors]


def test_written_tensors_raise_their_versions(ar, marshalling):
    """Every tensor that a call or a plan's start writes counts as changed in place, and no other one does."""
    torch = _torch()
    f = lambda n=300: torch.ones(n, device="cuda")                       # noqa: E731
    good = dict(step=1, lr=0.1)

    def changed(call, *tensors):
        before = versions(*tensors)
        call()
        return [a > b for a, b in zip(versions(*tensors), before)]

    p, g, m, v = f(), f(), f(), f()
    c = torch.zeros(300, dtype=torch.bfloat16, device="cuda")
    new = [f() for _ in range(3)]
    assert changed(lambda: ar.ar_adamw([p], [g], [m], [v], copies=[c], **good), p, g, m, v, c) == [1, 0, 1, 1, 1]
    assert changed(lambda: ar.ar_adamw([p], [g], [m], [v], out=[[t] for t in new], **good), p, g, m, v, *new) == \
        [0, 0, 0, 0, 1, 1, 1]
    plan = ar.ar_adamw_init([p], [g], [m], [v], copies=[c])
    assert changed(lambda: plan.start(**good), p, g, m, v, c) == [1, 0, 1, 1, 1]
    a, b = (ar.PackedState.zeros(300, "cuda") for _ in range(2))
    assert changed(lambda: ar.ar_adamw_packed([p], [g], [a], [b], seed=0, **good), p, g, *a, *b) == [1, 0, 1, 1, 1, 1]
    plan = ar.ar_adamw_packed_init([p], [g], [a], [b], out=([new[0]], [ar.PackedState.zeros(300, "cuda")], [b]))
    assert changed(lambda: plan.start(seed=0, **good), p, g, *a, *b, new[0]) == [0, 0, 0, 0, 1, 1, 1]
    out = f()
    assert changed(lambda: ar.ar_unpack_states([a], "exp_avg", outs=[out]), out, *a) == [1, 0, 0]
    norm = torch.zeros(1, device="cuda")
    assert changed(lambda: ar.ar_grad_norm([g], norm=norm), norm, g) == [1, 0]
    plan = ar.ar_grad_norm_init([g], norm=norm)
    assert changed(lambda: plan.start(), norm, g) == [1, 0]
    x, w, y, dy, dx, dg, db = (f().view(3, 100), f(100), f().view(3, 100), f().view(3, 100), f().view(3, 100), f(100),
                               f(100))
    assert changed(lambda: ar.ar_layer_norm([x], [w], ys=[y]), x, w, y) == [0, 0, 1]
    assert changed(lambda: ar.ar_layer_norm([x], [w], ys=[x]), x, w) == [1, 0]
    _, ms, rs = ar.ar_layer_norm([x], [w])
    assert changed(lambda: ar.ar_layer_norm_backward([dy], [x], [w], ms, rs, dxs=[dx], dgammas=[dg], dbetas=[db]),
                   x, w, dy, *ms, *rs, dx, dg, db) == [0, 0, 0, 0, 0, 1, 1, 1]
    # a refused call has written nothing
    with pytest.raises(ar.ArError):
        ar.ar_adamw([p], [g], [m], [v], step=1, lr=-1.0)
    assert changed(lambda: pytest.raises(ar.ArError, ar.ar_adamw, [p], [g], [m], [v], step=1, lr=-1.0), p, m, v) == \
        [0, 0, 0]


def test_stale_graphs_are_refused(ar, marshalling):
    """A backward pass through a parameter that a step has since replaced raises, as torch's own updates make it."""
    torch = _torch()
    for planned in (False, True):
        p = torch.nn.Parameter(torch.ones(8, 8, device="cuda"))
        g, m, v = (torch.ones(64, device="cuda") for _ in range(3))
        x = torch.ones(8, 8, device="cuda", requires_grad=True)
        loss = (x @ p).sum()
        if planned:
            ar.ar_adamw_init([p.view(64)], [g], [m], [v]).start(step=1, lr=0.1)
        else:
            ar.ar_adamw([p], [g], [m], [v], step=1, lr=0.1)
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="inplace operation"):
            loss.backward()
    with torch.inference_mode():           # such tensors have no counter, and need none
        p = torch.ones(8, device="cuda")
        ar.ar_adamw([p], [torch.ones(8, device="cuda")], [torch.zeros(8, device="cuda")],
                    [torch.zeros(8, device="cuda")], step=1, lr=0.5)
    ar.ar_adamw([p], [torch.ones(8, device="cuda")], [torch.zeros(8, device="cuda")],
                [torch.zeros(8, device="cuda")], step=1, lr=0.5)
    assert (p == 0).all()


@pytest.mark.parametrize("counts,launches", [([1] * 128, 1), ([1] * 129, 2), ([0, 8192] * 128, 1), ([0] * 200, 1),
                                             ([8193] * 64, 1), ([8193] * 64 + [1], 2), ([1 << 20], 1),
                                             ([(1 << 20) + 1], 2)])
def test_norm_plan_launches(ar, counts, launches):
    """One launch up to 128 tiles, of 8,192 elements and at least one a tensor that holds anything."""
    torch = _torch()
    rng = np.random.default_rng(len(counts))
    gs = [on_device(rng.standard_normal(n).astype(np.float32), "f32") for n in counts]
    plan = ar.ar_grad_norm_init(gs)
    assert plan.num_launches == ar.ar_update_num_launches(plan) == launches
    want = oracle.grad_norm([f64(g) for g in gs])
    for _ in range(2):
        assert abs(f64(plan.start())[0] - want) <= norm_bound(want)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_packed_large_form_agrees_with_the_small_one(ar, dtype):
    """2^24 elements take two vectors a thread: each tensor's parameters, codes and scales, over its whole length,
    are those of a smaller call that gives it the same number, and the oracle's in the second vector of a tile."""
    torch = _torch()
    odd = [70_001, 4096 + 2048 + 300, 4096 + 2047, 4096, 2049, 9]
    torch.manual_seed(5)
    rng = np.random.default_rng(5)
    config = dict(HYPER, seed=8)
    sets = []
    for last in ((1 << 24) - sum(odd), 7):
        sizes = odd + [last]
        if not sets:
            ps = [torch.randn(n, device="cuda").to(torch_dtype(dtype)) for n in sizes]
            gs = [torch.randn(n, device="cuda").to(torch_dtype(dtype)) for n in sizes]
            states = [packed_inputs(ar, rng, n, k % 5) for k, n in enumerate(odd)]
            ms, vs = ([s[i][0] for s in states] + [ar.PackedState.zeros(last, "cuda")] for i in (0, 1))
        sets.append(([p.clone()[:n] for p, n in zip(ps, sizes)], [g[:n] for g, n in zip(gs, sizes)],
                     *([ar.PackedState(s.codes.clone()[:n], s.scales.clone()[:oracle.blocks_of(n)])
                        for s, n in zip(x, sizes)] for x in (ms, vs))))
    assert sum(t.numel() for t in sets[0][0]) == 1 << 24
    for s in sets:
        ar.ar_adamw_packed(*s, **config)
    large, small = sets
    for k, n in enumerate(odd):
        assert torch.equal(large[0][k], small[0][k]), n
        for i in (2, 3):
            assert torch.equal(large[i][k].codes, small[i][k].codes), n
            assert torch.equal(large[i][k].scales, small[i][k].scales), n
        if n > 10_000:
            continue
        new = oracle.moments_f32(f32(gs[k]), states[k][0][1], states[k][1][1], HYPER["betas"], 1.0)
        bits = oracle.random_bits(8, k, n)
        for i, x, kind in ((2, new[0], "exp_avg"), (3, new[1], "exp_avg_sq")):
            codes, scales = oracle.pack(x, bits, kind)
            assert np.array_equal(large[i][k].scales.cpu().numpy(), scales), (n, kind)
            assert np.array_equal(large[i][k].codes.cpu().numpy(), codes), (n, kind)
        check_param(large[0][k], ps[k], gs[k], states[k][0][1], states[k][1][1], dtype)
