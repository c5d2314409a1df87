"""GPU parity of AdamW over a list of tensors and of its 8-bit moments with
the float64 oracle.

Tolerances are sums of roundings: with h = 2^-24 (half an fp32 step,
relative) every product, sum, square root and conversion adds one h of its
result.  8-bit codes and bf16 parameters are compared with the neighbours that
the oracle's value, moved by its tolerance either way, is rounded to.
"""

import math

import numpy as np
import pytest

from oracle import adamw as oa
from tests.gpu_util import cuda_or_skip

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
TINY = 2.0 ** -149  # an fp32 result below the normal range is off by half of this


@pytest.fixture(scope="module")
def torch():
    return cuda_or_skip()


@pytest.fixture(scope="module")
def bd():
    from matrix_inverse_roots_stack_b200 import binding
    return binding


def f64(t):
    return t.detach().double().cpu().numpy().ravel()


class Guarded:
    """Tensors cut from larger buffers at a given element offset, with bytes
    before and after that nobody may write."""

    def __init__(self, torch):
        self.torch, self.kept = torch, []

    def __call__(self, x, dtype, offset=0):
        torch = self.torch
        size = torch.empty((), dtype=dtype).element_size()
        n = x.numel()
        raw = torch.full((64 + offset + n + 64,), 0, dtype=dtype, device="cuda")
        raw.view(torch.uint8).fill_(0xA5)
        t = raw[64 + offset:64 + offset + n]
        t.copy_(x.reshape(-1))
        self.kept.append((raw, 64 + offset, n, size))
        return t.view(x.shape)

    def check(self):
        for raw, at, n, size in self.kept:
            b = raw.view(self.torch.uint8)
            assert bool((b[:at * size] == 0xA5).all()) and bool((b[(at + n) * size:] == 0xA5).all())


def spread(torch, gen, n, std):
    """Values whose scale differs from run to run of 100."""
    x = torch.randn(n, generator=gen) * std
    s = torch.exp(1.5 * torch.randn(-(-n // 100) if n else 0, generator=gen))
    return x * s.repeat_interleave(100)[:n]


SIZES = [(0,), (1,), (7,), (31,), (255,), (256,), (257,), (33, 65), (2048,), (2049,), (3, 5, 700), ()]


def make(torch, bd, sizes, bits, param, grad, copy, offsets, seed=0, hp=None, decay=0.1, lr_scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    g = Guarded(torch)
    P, G, C, M, V, S = [], [], [], [], [], []
    for i, shape in enumerate(sizes):
        offset = offsets[i % len(offsets)] if isinstance(offsets, list) else offsets
        n = int(np.prod(shape))
        P.append(g((torch.randn(n, generator=gen) * 0.02).view(shape), param, offset))
        G.append(g(torch.zeros(shape), grad, offset))
        C.append(g(torch.zeros(shape), copy, offset) if copy is not None else None)
        code = torch.uint8 if bits == 8 else torch.float32
        M.append(g(torch.zeros(n), code, offset))
        V.append(g(torch.zeros(n), code, offset))
        S.append([g(torch.zeros(-(-n // 256)), torch.uint8, offset) for _ in "mv"] if bits == 8 else [None, None])
    opt = bd.AdamW(P, G, hp=hp, copies=C if copy is not None else None, state_bits=bits, m=M, v=V,
                   m_scale=[s[0] for s in S], v_scale=[s[1] for s in S], weight_decay=decay, lr_scale=lr_scale)
    return opt, g, gen


def moments_of(opt, i):
    if opt.state_bits[i] == 32:
        return f64(opt.m[i]), f64(opt.v[i])
    r = oa.decode(opt.v[i].cpu().numpy(), opt.v_scale[i].cpu().numpy(), oa.V_FORMAT)
    return oa.decode(opt.m[i].cpu().numpy(), opt.m_scale[i].cpu().numpy(), oa.M_FORMAT), r * r


def snapshot(opt):
    return [(f64(opt.params[i]), f64(opt.grads[i]), *moments_of(opt, i)) for i in range(len(opt.params))]


def between(got, x, err, fmt, u, exponents):
    """got is what some value within err of x is held as."""
    lo = oa.held(np.maximum(np.abs(x) - err, 0), fmt, exponents, u)
    hi = oa.held(np.abs(x) + err, fmt, exponents, u)
    if fmt is oa.M_FORMAT:
        zero = np.abs(x) <= err  # the sign is open there
        assert np.all(zero | (np.sign(got) == np.sign(x)) | (got == 0))
        got = np.abs(got)
    assert np.all((lo <= got) & (got <= hi))
    sure = err <= 1e-5 * np.abs(x)  # where v is below fp32's normal range the tolerance spans many codes
    return np.mean((got == oa.held(np.abs(x), fmt, exponents, u))[sure]) if sure.any() else 1.0


def check_step(torch, opt, before, t, lr, coef=1.0, decay=0.1, lr_scale=1.0):
    """One step's results against the oracle's from the state before it."""
    hp, f32 = opt.hp, np.float32
    lr = float(f32(f32(lr) * f32(lr_scale)))
    decay, coef = float(f32(decay)), float(f32(coef))
    b1, b2, eps = hp.beta1, hp.beta2, hp.adam_eps
    same = []
    for i, (p0, g, m0, v0) in enumerate(before):
        if not len(p0):
            continue
        p, m, v = oa.step(p0, g, m0, v0, t, b1, b2, eps, lr, decay, coef)
        # m: product and sum on one side, coef, product and sum on the other
        em = H * (2 * np.abs(b1 * m0) + 3 * np.abs((1 - b1) * coef * g)) * 1.01 + 2 * TINY
        # v: at most five roundings of positive terms; its root half of that and the approximate square root's
        # 2^-23; below fp32's normal range v counts as 0
        ev, r = 5 * H * v * 1.01 + 2 * TINY, np.sqrt(v)
        er = np.where(v < 1.01 * 2.0 ** -126, r, 4.5 * H * r * 1.01)
        c1, c2 = 1 / (1 - b1 ** t), 1 / np.sqrt(1 - b2 ** t)
        den = r * c2 + eps
        ratio = np.abs(m * c1 / den)
        # update: c1, product, division (two steps), and the denominator's root, c2, product and sum; then the
        # decay's product, the sum, the learning rate's and the last sum
        ed = ratio * 12 * H + c1 * em / den + ratio * c2 * er / den
        ep = lr * (ed + 4 * H * (ratio + decay * np.abs(p0))) + H * np.abs(p) * 1.01 + TINY
        got = f64(opt.params[i])
        dm, dv, dp = oa.draws(hp.seed, t, i, np.arange(len(p)))
        if opt.params[i].dtype == torch.float32:
            assert np.all(np.abs(got - p) <= ep), (i, np.max(np.abs(got - p) / ep))
            if opt.copies[i] is not None:  # the new value rounded once more, to nearest
                assert torch.equal(opt.copies[i], opt.params[i].to(opt.copies[i].dtype))
        else:
            lo = oa.on_grid(np.maximum(np.abs(p) - ep, 0), oa.BF16_FORMAT, dp)
            hi = oa.on_grid(np.abs(p) + ep, oa.BF16_FORMAT, dp)
            assert np.all((lo <= np.abs(got)) & (np.abs(got) <= hi))
            assert np.all((np.sign(got) == np.sign(p)) | (np.abs(p) <= ep) | (got == 0))
            same.append(np.mean(np.abs(got) == oa.on_grid(p, oa.BF16_FORMAT, dp)))
        gm, gv = moments_of(opt, i)
        if opt.state_bits[i] == 32:
            assert np.all(np.abs(gm - m) <= em) and np.all(np.abs(gv - v) <= ev)
            continue
        for x, e, fmt, scale, u, got in ((m, em, oa.M_FORMAT, opt.m_scale[i], dm, gm),
                                         (r, er, oa.V_FORMAT, opt.v_scale[i], dv, np.sqrt(gv))):
            s = scale.cpu().numpy().astype(int) - 127
            assert np.all(s >= oa.block_exponents(np.maximum(np.abs(x) - e, 0), fmt))
            assert np.all(s <= oa.block_exponents(np.abs(x) + e, fmt))
            same.append(between(got, x, e, fmt, u, s))
    # rounding to the oracle's own neighbour fails only where the tolerance reaches over a border
    assert all(x > 0.98 for x in same) and (not same or np.mean(same) > 0.999)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [0, 1, 4, 8, 16])
@pytest.mark.parametrize("param,grad,copy", [("float32", "float32", None), ("float32", "bfloat16", "bfloat16"),
                                             ("float32", "float16", "float16"), ("bfloat16", "bfloat16", None),
                                             ("bfloat16", "float32", None), ("bfloat16", "float16", None)])
def test_steps_match_the_oracle(torch, bd, bits, offset, param, grad, copy):
    ty = lambda s: getattr(torch, s) if s else None
    hp = bd.make_adamw_hparams(seed=77 + (5 << 32))
    opt, guard, gen = make(torch, bd, SIZES, bits, ty(param), ty(grad), ty(copy), offset, hp=hp)
    for t in range(1, 5):
        for g in opt.grads:
            g.copy_(spread(torch, gen, g.numel(), 1e-2).view(g.shape))
        before = snapshot(opt)
        opt.step(1e-3)
        check_step(torch, opt, before, t, 1e-3)
        assert opt.status() == (0, 0)
    assert opt.steps_taken() == 4
    guard.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,copy", [("float32", "float32", None), ("float32", "bfloat16", "float16"),
                                             ("float32", "float16", "bfloat16"), ("bfloat16", "bfloat16", None),
                                             ("bfloat16", "float32", None), ("bfloat16", "float16", None)])
def test_steps_of_longer_lists_match_the_oracle(torch, bd, bits, param, grad, copy):
    # more tiles than SMs: these go through the ring, whole tiles staged, others not
    ty = lambda s: getattr(torch, s) if s else None
    hp = bd.make_adamw_hparams(seed=78)
    opt, guard, gen = make(torch, bd, [(4096 * 130 + 777,)] + SIZES + [(4096 * 25,), (4096 * 20 + 1,)], bits, ty(param),
                           ty(grad), ty(copy), [0, 1, 4, 16, 0, 8, 0], hp=hp)
    for t in range(1, 3):
        for g in opt.grads:
            g.copy_(spread(torch, gen, g.numel(), 1e-2).view(g.shape))
        before = snapshot(opt)
        opt.step(1e-3)
        check_step(torch, opt, before, t, 1e-3)
        assert opt.status() == (0, 0)
    guard.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e3, 1e15])
def test_gradient_magnitudes(torch, bd, bits, scale):
    # squares from below fp32's range (they vanish: r = 0) to near its end; a block with one value 1e6 times the
    # others keeps them apart from zero in r
    hp = bd.make_adamw_hparams(adam_eps=1e-8, seed=3)
    opt, guard, gen = make(torch, bd, [(700,), (256,)], bits, torch.float32, torch.float32, None, 0, hp=hp)
    for t in range(1, 4):
        for g in opt.grads:
            g.copy_(torch.randn(g.shape, generator=gen) * scale)
            g[3] = 1e6 * scale if scale < 1e12 else scale
        before = snapshot(opt)
        opt.step(1e-2)
        check_step(torch, opt, before, t, 1e-2)
    if bits == 8 and scale > 1e-15:
        for i in range(2):
            assert bool((opt.v[i][opt.grads[i] != 0] > 0).all())
    guard.check()


def test_no_gradient_leaves_zero_moments(torch, bd):
    for bits in (32, 8):
        opt, guard, _ = make(torch, bd, [(600,)], bits, torch.float32, torch.float32, None, 0, decay=0.0)
        p = opt.params[0].clone()
        for _ in range(3):
            opt.step(0.1)
        assert torch.equal(p, opt.params[0]) and opt.status() == (0, 0)
        m, v = opt.read_moments()
        assert not bool(m.any()) and not bool(v.any())
        guard.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_scalar_and_vector_accesses_give_the_same_bits(torch, bd, bits):
    out = []
    for offset in (0, 1, 4, 16):
        opt, guard, gen = make(torch, bd, SIZES + [(9000,), (4096 * 160 + 9,)], bits, torch.bfloat16, torch.bfloat16, None, offset)
        for _ in range(3):
            for g in opt.grads:
                g.copy_(spread(torch, gen, g.numel(), 1e-2).view(g.shape))
            opt.step(1e-2)
        out.append([t.clone() for t in opt.params + opt.m + opt.v + opt.m_scale + opt.v_scale if t is not None])
        guard.check()
    assert all(torch.equal(a, b) for other in out[1:] for a, b in zip(out[0], other))


def test_list_of_both_moment_widths_and_settings_for_each(torch, bd):
    # 8-bit and 32-bit tensors, types, decays and rates side by side; each tensor as in a list of its own kind
    gen = torch.Generator().manual_seed(5)
    shapes, bits = [(5000,), (64,), (300, 20), (1,)], [8, 32, 8, 32]
    types = [torch.float32, torch.float32, torch.bfloat16, torch.bfloat16]
    P = [(torch.randn(s, generator=gen) * 0.1).to(t).cuda() for s, t in zip(shapes, types)]
    G = [torch.randn(s, generator=gen).cuda() for s in shapes]
    copies = [torch.zeros(5000, dtype=torch.bfloat16, device="cuda"), None, None, None]
    decay, rate = [0.1, 0.0, 0.01, 0.5], [1.0, 0.5, 0.0, 2.0]
    opt = bd.AdamW(P, G, copies=copies, state_bits=bits, weight_decay=decay, lr_scale=rate)
    for t in (1, 2):
        before = snapshot(opt)
        opt.step(1e-2)
        for i in range(4):
            one = [(np.zeros(0),) * 4] * 4
            one[i] = before[i]
            check_step(torch, opt, one, t, 1e-2, decay=decay[i], lr_scale=rate[i])


def test_large_lists_take_larger_chunks(torch, bd):
    # over 2^28 elements a chunk is four times as long: the ends of tensors and what lies around element 2^28
    n = (1 << 28) + 1003
    P = [torch.full((n,), 1.0, dtype=torch.bfloat16, device="cuda"), torch.ones(777, device="cuda")]
    G = [torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1)),
         torch.ones(777, device="cuda")]
    opt = bd.AdamW(P, G, state_bits=8, weight_decay=0.1)
    opt.step(1e-2)
    assert opt.status() == (0, 0)
    check_slices(torch, opt, [(0, 3000), (8192 - 256, 8192 + 256), ((1 << 28) - 512, 1 << 28), (n - n % 256, n)])
    check_step(torch, opt, [(np.zeros(0),) * 4, (np.ones(777), np.ones(777), np.zeros(777), np.zeros(777))], 1, 1e-2)


def check_slices(torch, opt, spans):
    """First steps of tensor 0, all ones and zero moments before, on slices that start at a block."""
    for a, b in spans:
        g = f64(opt.grads[0][a:b])
        p, m, v = oa.step(1.0, g, 0.0, 0.0, 1, opt.hp.beta1, opt.hp.beta2, opt.hp.adam_eps, float(np.float32(1e-2)),
                          float(np.float32(0.1)))
        dm, dv, dp = oa.draws(opt.hp.seed, 1, 0, np.arange(a, b, dtype=np.uint64))
        got = f64(opt.params[0][a:b])
        e = 40 * H  # |p| is about 1, and the update a hundredth of it
        assert np.all((got >= oa.on_grid(p - e, oa.BF16_FORMAT, dp)) & (got <= oa.on_grid(p + e, oa.BF16_FORMAT, dp)))
        s = slice(a // 256, -(-b // 256))
        for x, code, scale, fmt, u in ((m, opt.m, opt.m_scale, oa.M_FORMAT, dm),
                                       (np.sqrt(v), opt.v, opt.v_scale, oa.V_FORMAT, dv)):
            sc = scale[0][s].cpu().numpy()
            got = oa.decode(code[0][a:b].cpu().numpy(), sc, fmt)
            between(got, x, 5 * H * np.abs(x), fmt, u, sc.astype(int) - 127)


def test_element_offsets_beyond_32_bits(torch, bd):
    n = (1 << 32) + 5003
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    P = torch.full((n,), 1.0, dtype=torch.bfloat16, device="cuda")
    G = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
    opt = bd.AdamW([P], [G], state_bits=8, weight_decay=0.1)
    clip = bd.GradClip([G])
    opt.step(1e-2)
    assert opt.status() == (0, 0)
    check_slices(torch, opt, [(0, 1024), ((1 << 31) - 256, (1 << 31) + 256), ((1 << 32) - 512, (1 << 32) + 512),
                              (n - n % 256, n)])
    # the norm of n ones; each block's sum of squares is a whole number
    G.fill_(1.0)
    assert clip.norm()[0].item() == np.float32(np.sqrt(float(n)))


# ---------------------------------------------------------------- the step number, scalars on the device

@pytest.mark.parametrize("bits", [32, 8])
def test_explicit_and_counted_steps_agree(torch, bd, bits):
    out = []
    for explicit in (False, True):
        opt, _, gen = make(torch, bd, [(5000,)], bits, torch.float32, torch.float32, None, 0)
        for t in range(1, 30):
            opt.grads[0].copy_(torch.randn(5000, generator=gen))
            opt.step(1e-2, step=t if explicit else 0)
        assert opt.steps_taken() == 29
        out.append([opt.params[0].clone(), opt.m[0].clone(), opt.v[0].clone()])
    # the counter multiplies beta^t up where the host raises to the power: in double the two differ by far less
    # than an fp32 step, so c1 and c2 may round differently once in many millions of steps, and not here
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_resumed_from_a_checkpoint(torch, bd):
    # moments and counter carried into a new list: 32-bit moments exactly
    a, _, gen = make(torch, bd, SIZES, 32, torch.float32, torch.float32, None, 0)
    grads = [[torch.randn(g.shape, generator=gen) for g in a.grads] for _ in range(6)]

    def run(opt, gs):
        for step in gs:
            for g, x in zip(opt.grads, step):
                g.copy_(x)
            opt.step(1e-2)

    run(a, grads[:3])
    m, v = a.read_moments()
    b = bd.AdamW([p.clone() for p in a.params], [g.clone() for g in a.grads], weight_decay=0.1,
                 steps_taken=a.steps_taken())
    b.load_moments(m, v)
    assert b.status() == (0, 0)
    run(a, grads[3:])
    run(b, grads[3:])
    assert all(torch.equal(x, y) for x, y in zip(a.params + a.m + a.v, b.params + b.m + b.v))
    assert b.steps_taken() == 6


def test_learning_rate_and_coefficient_on_the_device(torch, bd):
    opts = [make(torch, bd, [(3000,)], 32, torch.float32, torch.float32, None, 0)[0] for _ in range(2)]
    lr, coef = torch.tensor(0.125, device="cuda"), torch.tensor([0.25], device="cuda")
    for o in opts:
        o.grads[0].copy_(torch.linspace(-1, 1, 3000))
    opts[1].grads[0].mul_(0.25)  # exact
    opts[0].step(lr, coef=coef)
    opts[1].step(0.125)
    assert torch.equal(opts[0].params[0], opts[1].params[0]) and torch.equal(opts[0].v[0], opts[1].v[0])


@pytest.mark.parametrize("bits", [32, 8])
def test_step_is_not_taken_where_the_coefficient_is_not_finite(torch, bd, bits):
    opt, guard, gen = make(torch, bd, SIZES, bits, torch.float32, torch.float32, torch.bfloat16, 0)
    coef = torch.ones(1, device="cuda")

    def state():
        return [t.clone() for t in opt.params + opt.copies + opt.m + opt.v + opt.m_scale + opt.v_scale
                if t is not None]

    for g in opt.grads:
        g.copy_(torch.randn(g.shape, generator=gen))
    opt.step(1e-2, coef=coef)
    assert opt.status()[0] == 0
    kept = state()
    for bad in (float("nan"), float("inf"), -float("inf")):
        coef.fill_(bad)
        opt.step(1e-2, coef=coef)
        assert opt.status() == (bd.SHAMPOO_ENONFINITE, 1)
        opt.step(1e-2, coef=coef, step=9)
        assert opt.steps_taken() == 1
        assert all(torch.equal(a, b) for a, b in zip(kept, state()))
    coef.fill_(1.0)
    before = snapshot(opt)
    opt.step(1e-2, coef=coef)
    assert opt.status() == (0, 0) and opt.steps_taken() == 2
    check_step(torch, opt, before, 2, 1e-2)
    guard.check()


def test_non_finite_gradients_without_a_coefficient(torch, bd):
    # 32 bits: the elements concerned follow IEEE arithmetic; 8 bits: their blocks of 256
    for bits in (32, 8):
        opt, guard, gen = make(torch, bd, [(1024,), (100,)], bits, torch.float32, torch.float32, None, 0)
        for g in opt.grads:
            g.copy_(torch.randn(g.shape, generator=gen))
        opt.grads[0][300] = float("nan")
        opt.grads[0][800] = float("inf")
        opt.step(1e-2)
        assert opt.status() == (bd.SHAMPOO_ENONFINITE, 1)
        m, _ = opt.read_moments()
        bad = ~torch.isfinite(opt.views(m)[0])
        want = torch.zeros(1024, dtype=torch.bool, device="cuda")
        if bits == 32:
            want[300] = want[800] = True
        else:
            want[256:512] = want[768:1024] = True
            assert opt.m_scale[0].tolist()[1::2] == [255, 255] and opt.v_scale[0].tolist()[1::2] == [255, 255]
        assert torch.equal(bad, want)
        assert bool(torch.isfinite(opt.params[1]).all())
        assert torch.isfinite(opt.params[0]).sum() >= 1022
        # the bit is that of the last call
        opt2, _, _ = make(torch, bd, [(64,)], bits, torch.float32, torch.float32, None, 0)
        opt2.grads[0].fill_(float("nan"))
        opt2.step(1e-2, coef=torch.full((1,), float("nan"), device="cuda"))
        opt2.grads[0].fill_(1.0)
        opt2.step(1e-2)
        assert opt2.status() == (0, 0)
        guard.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad", [("float32", "float32"), ("float32", "bfloat16"), ("bfloat16", "float32"),
                                        ("bfloat16", "bfloat16")])
@pytest.mark.parametrize("n,offset", [(1500, 0), (1500, 1), (4096 * 160 + 9, 0), (4096 * 160 + 9, 1)])
def test_gradients_whose_square_overflows(torch, bd, bits, param, grad, n, offset):
    # finite gradients, infinite second moments: sqrt(inf) = inf, m / inf = 0, and only the decay moves the parameter.
    # In 8 bits v is infinite for the block from the next step on.  Short lists and long ones, which go through the ring
    opt, guard, gen = make(torch, bd, [(n,)], bits, getattr(torch, param), getattr(torch, grad), None, offset, seed=9)
    big = [3, 700, 702, 1499] if n < 4096 else [3, 700, 4096 * 100 + 255, 4096 * 160 - 1, n - 1]
    over = np.zeros(n, bool)
    over[big] = True
    lr, decay = float(np.float32(1e-2)), float(np.float32(0.1))
    frozen = over
    for t in range(1, 4):
        opt.grads[0].copy_(torch.randn(n, generator=gen))
        if t == 1:
            for i, x in zip(big, (1e21, -1e30, 6e20, -3e21, 2e25)):
                opt.grads[0][i] = x
        before = snapshot(opt)
        opt.step(1e-2)
        assert opt.status() == (bd.SHAMPOO_ENONFINITE, 1)
        p0, got = before[0][0], f64(opt.params[0])
        p = p0 - lr * decay * p0
        e = 3 * H * (np.abs(p) + lr * decay * np.abs(p0))  # product, sum and last sum, each of them one rounding
        if param == "float32":
            assert np.all(np.abs(got - p)[frozen] <= e[frozen])
        else:
            dp = oa.draws(opt.hp.seed, t, 0, np.arange(n))[2]
            lo, hi = (oa.on_grid(np.maximum(np.abs(p) + s * e, 0), oa.BF16_FORMAT, dp) for s in (-1, 1))
            assert np.all(((lo <= np.abs(got)) & (np.abs(got) <= hi))[frozen])
        assert np.isfinite(got).all()
        other = [np.where(frozen, 0.0, x) for x in before[0]]  # the others as ever
        if t == 1:
            P, g, m, v = other
            want, _, _ = oa.step(P, g, m, v, 1, opt.hp.beta1, opt.hp.beta2, opt.hp.adam_eps, lr, decay)
            tol = lr * 30 * H + 1.01 * (H if param == "float32" else 2.0 ** -7) * np.abs(want)
            assert np.all(np.abs(got - want)[~frozen] <= tol[~frozen])
        if bits == 8:
            frozen = np.repeat(np.add.reduceat(over, np.arange(0, n, 256)) > 0, 256)[:n]
            assert np.array_equal(opt.v_scale[0].cpu().numpy() == 255, frozen[::256])
            assert not bool((opt.m_scale[0] == 255).any())
        m, v = (f64(opt.views(x)[0]) for x in opt.read_moments())
        assert np.isfinite(m).all() and np.array_equal(v == np.inf, frozen) and not np.isnan(v).any()
    guard.check()


def test_bf16_parameters_stay_infinite_or_nan(torch, bd):
    P = [torch.tensor([float("inf"), -float("inf"), float("nan"), 1.0], dtype=torch.bfloat16, device="cuda")]
    G = [torch.zeros(4, device="cuda")]
    opt = bd.AdamW(P, G, weight_decay=0.0)
    for _ in range(20):
        opt.step(1e-3)
    p = P[0].float().cpu().numpy()
    # an infinite parameter times a decay of zero is not a number
    assert np.isnan(p[:3]).all() and p[3] == 1.0


# ---------------------------------------------------------------- stochastic rounding

def test_second_moment_follows_slow_changes(torch, bd):
    # v decays by 0.1% a step: rounding to nearest would never move it.  After 2000 steps without gradients it is
    # beta2^2000 = 0.135 of its start.  Each element's root performs a random walk of 2000 roundings, each of
    # variance at most w^2/4 for a code of width w <= r/16 .. r/32 taken with probability about 0.0005 r/w: a
    # step's variance is about w * 0.0005 r <= r^2 * 3.2e-5, 2000 of them 0.063 r^2; the mean over 65536
    # elements has a deviation of at most sqrt(0.063 / 65536) = 1e-3 (relative); 6 of them
    n = 65536
    opt = bd.AdamW([torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")], state_bits=8)
    r0 = torch.rand(opt.moment_elems, device="cuda", generator=torch.Generator("cuda").manual_seed(3)) + 0.5
    opt.load_moments(torch.zeros_like(r0), r0 * r0)
    before = opt.read_moments()[1].sqrt().double().mean().item()
    for _ in range(2000):
        opt.step(0.0)
    after = opt.read_moments()[1].sqrt().double().mean().item()
    assert abs(after / (before * 0.999 ** 1000) - 1) < 6e-3


def test_bf16_parameters_collect_small_updates(torch, bd):
    # 512 updates of 1e-5 beside a bf16 step of 2^-7 at 1: to nearest, none would count.  Each is a Bernoulli draw
    # of probability 1e-5 * 128 = 1.3e-3 (x 2 below 1); the mean over 2^18 parameters deviates by
    # sqrt(512 * 1e-5 * 2^-8 / 2^18) = 8.7e-6; 6 of them, and 1% for the moments' start (g is constant, so the
    # update is lr at every step)
    n = 1 << 18
    P = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    opt = bd.AdamW([P], [torch.ones(n, device="cuda")])
    for _ in range(512):
        opt.step(1e-5)
    assert abs((1 - P.double()).mean().item() - 512e-5) < 6 * 8.7e-6 + 1e-5


# ---------------------------------------------------------------- moments in and out

@pytest.mark.parametrize("offset", [0, 1, 4, 16])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_moments_in_and_out(torch, bd, offset, dtype):
    opt, guard, gen = make(torch, bd, SIZES, 8, torch.float32, torch.float32, None, offset)
    sizes = [p.numel() for p in opt.params]
    assert opt.moment_elems == sum(-(-n // 256) * 256 for n in sizes)
    flat = [torch.full((opt.moment_elems,), float("nan"), device="cuda") for _ in "mv"]  # tails are not read
    for a, b, n in zip(opt.views(flat[0]), opt.views(flat[1]), sizes):
        a.copy_(spread(torch, gen, n, 1e-3).view(a.shape))
        b.copy_(spread(torch, gen, n, 1e-3).square().view(b.shape))
    opt.load_moments(*flat)
    assert opt.status() == (0, 0)
    out = opt.read_moments(getattr(torch, dtype))
    for i, n in enumerate(sizes):
        if not n:
            continue
        m, v = f64(opt.views(flat[0])[i]), f64(opt.views(flat[1])[i])
        r = np.sqrt(v.astype(np.float32)).astype(np.float64)  # the root is rounded to fp32 first
        em, er = oa.block_exponents(m, oa.M_FORMAT), oa.block_exponents(r, oa.V_FORMAT)
        assert np.array_equal(opt.m_scale[i].cpu().numpy().astype(int) - 127, em)
        assert np.array_equal(opt.v_scale[i].cpu().numpy().astype(int) - 127, er)
        hm, hr = oa.held(m, oa.M_FORMAT, em), oa.held(r, oa.V_FORMAT, er)
        to = lambda x: torch.from_numpy(x.astype(np.float32)).to(getattr(torch, dtype))
        assert torch.equal(opt.views(out[0])[i].cpu().ravel(), to(hm))
        assert torch.equal(opt.views(out[1])[i].cpu().ravel(), to(hr * hr))
    tails = torch.ones(opt.moment_elems, dtype=torch.bool)
    for t in opt.views(tails):
        t.fill_(False)
    for x in out:
        assert not bool(x.cpu()[tails].any())
    # what was read is held exactly (a block whose maximum was rounded down to the format's largest number takes
    # the scale below, where its numbers are found again)
    if dtype == "float32":
        opt.load_moments(*out)
        assert all(torch.equal(a, b) for a, b in zip(out, opt.read_moments()))
    guard.check()


def test_moments_of_extreme_size(torch, bd):
    opt = bd.AdamW([torch.zeros(256 * 6, device="cuda")], [torch.zeros(256 * 6, device="cuda")], state_bits=8)
    m, v = torch.zeros(256 * 6, device="cuda"), torch.zeros(256 * 6, device="cuda")
    fmax, fmin = torch.finfo(torch.float32).max, 2.0 ** -149
    m[0], m[1], v[0], v[1] = fmax, -1.0, fmax, 1e-20
    m[256], m[257], v[256], v[257] = fmin, -fmin, fmin, 0.0
    m[512], m[513], v[512] = 448.0, 2.0 ** -9, 31744.0 ** 2
    m[768], v[768] = 448.0 + 2.0 ** -15, 31744.0 ** 2 + 64.0 * 2  # the next fp32 numbers, and one more
    m[1024], v[1024] = 2.0 ** -127, 2.0 ** -126
    opt.load_moments(m, v)
    assert opt.status() == (0, 0)
    r = v.sqrt()
    for x, got_s, got, fmt in ((m, opt.m_scale, opt.m, oa.M_FORMAT), (r, opt.v_scale, opt.v, oa.V_FORMAT)):
        e = oa.block_exponents(f64(x), fmt)
        assert np.array_equal(got_s[0].cpu().numpy().astype(int) - 127, e)
        # an element more than 2^126 below its block's largest vanishes on the way
        assert np.array_equal(np.abs(oa.decode(got[0].cpu().numpy(), e + 127, fmt)), np.abs(oa.held(f64(x), fmt, e)))
    m.zero_()
    m[300], v[600] = float("nan"), -1.0  # no moment is negative
    opt.load_moments(m, v)
    assert opt.status() == (bd.SHAMPOO_ENONFINITE, 1)
    assert opt.m_scale[0].tolist()[1] == 255 and opt.v_scale[0].tolist()[2] == 255


@pytest.mark.parametrize("offset", [0, 1])
def test_infinite_second_moments_loaded_freeze_their_block(torch, bd, offset):
    # the block reads back as infinite, zeros in it too, and its parameters have no update but the decay
    opt, guard, gen = make(torch, bd, [(700,)], 8, torch.float32, torch.float32, None, offset, decay=0.5)
    m, v = torch.zeros(768, device="cuda"), torch.zeros(768, device="cuda")
    v[300] = float("inf")
    opt.load_moments(m, v)
    assert opt.status() == (bd.SHAMPOO_ENONFINITE, 1) and opt.v_scale[0].tolist() == [1, 255, 1]
    assert torch.equal(opt.views(opt.read_moments()[1])[0] == float("inf"), torch.arange(700, device="cuda") // 256 == 1)
    opt.grads[0].fill_(1.0)
    p0 = f64(opt.params[0])
    opt.step(0.125)
    got = f64(opt.params[0])
    want = p0 * (1 - 0.125 * 0.5)
    assert np.all(np.abs(got - want)[256:512] <= 3 * H * np.abs(p0)[256:512])
    assert np.all(np.abs(got - (want - 0.125))[np.r_[0:256, 512:700]] <= 0.125 * 30 * H + 1e-8)  # g / (|g| + eps)
    guard.check()


# ---------------------------------------------------------------- graphs and streams

@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_replays(torch, bd, bits):
    ref, _, gen = make(torch, bd, [(5000,), (77,)], bits, torch.bfloat16, torch.bfloat16, None, 0)
    opt, guard, _ = make(torch, bd, [(5000,), (77,)], bits, torch.bfloat16, torch.bfloat16, None, 0)
    clips = [bd.GradClip(o.grads) for o in (ref, opt)]
    lr = torch.zeros((), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # the first call already
        opt.step(lr, coef=clips[1].norm(1.0)[1:])
    for t in range(6):
        lr.fill_(1e-2 / (t + 1))
        for a, b in zip(ref.grads, opt.grads):
            a.copy_(torch.randn(a.shape, generator=gen))
            b.copy_(a)
        ref.step(lr, coef=clips[0].norm(1.0)[1:])
        graph.replay()
    assert ref.status() == (0, 0) and opt.status() == (0, 0) and opt.steps_taken() == 6
    assert all(torch.equal(a, b) for a, b in zip(ref.params + ref.m + ref.v, opt.params + opt.m + opt.v))
    # two graphs of one list, replayed in turn, share its counter
    second = torch.cuda.CUDAGraph()
    with torch.cuda.graph(second):
        opt.step(lr, coef=clips[1].norm(1.0)[1:])
    graph.replay()
    second.replay()
    for _ in range(2):
        ref.step(lr, coef=clips[0].norm(1.0)[1:])
    assert opt.steps_taken() == 8
    assert all(torch.equal(a, b) for a, b in zip(ref.params + ref.m + ref.v, opt.params + opt.m + opt.v))
    guard.check()


def test_captured_with_an_explicit_step_number(torch, bd):
    a, _, gen = make(torch, bd, [(3000,)], 8, torch.float32, torch.float32, None, 0)
    b, _, _ = make(torch, bd, [(3000,)], 8, torch.float32, torch.float32, None, 0)
    a.grads[0].copy_(torch.randn(3000, generator=gen))
    b.grads[0].copy_(a.grads[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(1e-2, step=7)
    for _ in range(2):
        a.step(1e-2, step=7)
        graph.replay()
    assert torch.equal(a.params[0], b.params[0]) and torch.equal(a.m[0], b.m[0]) and b.steps_taken() == 7


def test_construction_is_refused_while_capturing(torch, bd):
    p, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    opt = bd.AdamW([p], [g])
    ws = torch.empty(opt.ws.numel(), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stream = torch.cuda.current_stream().cuda_stream
        rc = bd.load().shampoo_adamw_bind(opt._ctx, 0, ws.data_ptr(), ws.numel(), stream)
        opt.step(0.0)
    assert rc == bd.SHAMPOO_EINVAL
    graph.replay()
    assert opt.status() == (0, 0)


def test_lists_on_two_streams(torch, bd):
    # two lists stepped at the same time, on streams other than the one that made them
    pair = [make(torch, bd, [(700000,), (1003,)], 8, torch.bfloat16, torch.bfloat16, None, 0, seed=s) for s in (1, 1)]
    ref = make(torch, bd, [(700000,), (1003,)], 8, torch.bfloat16, torch.bfloat16, None, 0, seed=1)[0]
    x = [torch.randn(g.shape, generator=pair[0][2]) for g in ref.grads]
    for o in (ref, pair[0][0], pair[1][0]):
        for g, y in zip(o.grads, x):
            g.copy_(y)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(50):
        ref.step(1e-2)
        for (o, _, _), s in zip(pair, streams):
            o.step(1e-2, stream=s)
    torch.cuda.synchronize()
    for (o, guard, _), s in zip(pair, streams):
        assert o.status(s) == (0, 0) and o.steps_taken(s) == 50
        assert all(torch.equal(a, b) for a, b in zip(ref.params + ref.m + ref.v, o.params + o.m + o.v))
        guard.check()


def test_memory_is_not_handed_out_while_a_stream_uses_it(torch, bd):
    # tensors of the current stream, stepped on another one that is behind; then everything is dropped
    side, n = torch.cuda.Stream(), 300000
    for own in (False, True):  # moments made by the caller, or by the list
        p, g = torch.ones(n, device="cuda"), torch.ones(n, device="cuda")
        m = v = None
        if own:
            m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        opt, clip = bd.AdamW([p], [g], m=m, v=v), bd.GradClip([g])
        clip.clip(1.0)  # both are loaded then
        opt.step(1e-3)
        torch.cuda.synchronize()
        used = {t.data_ptr() for t in [p, g] + opt.m + opt.v}
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # 0.1 s
            clip.clip(1.0)
            opt.step(1e-3)
        del p, g, m, v, opt, clip
        new = [torch.empty(n, device="cuda") for _ in range(8)]
        assert not side.query(), "the stream has to be behind still"
        assert not used & {t.data_ptr() for t in new}
        torch.cuda.synchronize()
        del new


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_moments_read_and_loaded_on_another_stream(torch, bd, dtype):
    # the current stream is behind, with a dropped temporary of the outputs' size still in its use
    n, side, dtype = 300000, torch.cuda.Stream(), getattr(torch, dtype)
    opt = bd.AdamW([torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")], state_bits=8)
    m = torch.randn(opt.moment_elems, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    v = m.square()
    opt.load_moments(m, v)
    want = opt.read_moments(dtype)
    doubled = [t * 2 for t in want]
    temps = [torch.full((opt.moment_elems,), 5.0, dtype=dtype, device="cuda") for _ in "mv"]
    torch.cuda.synchronize()  # every kernel has run once: loading one would wait for the device
    torch.cuda._sleep(200_000_000)  # 0.1 s
    for t in temps:
        t.fill_(7.0)
    used = {t.data_ptr() for t in temps}
    del temps, t
    opt.load_moments(m, v, stream=side)
    got = opt.read_moments(dtype, stream=side)
    assert not torch.cuda.current_stream().query(), "the stream has to be behind still"
    assert not used & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert opt.status(side) == (0, 0) and all(torch.equal(a, b) for a, b in zip(got, want))
    # dropped while the current stream still reads them: not handed out again on their own stream
    torch.cuda._sleep(200_000_000)
    kept = [t * 2 for t in got]
    used = {t.data_ptr() for t in got}
    del got
    with torch.cuda.stream(side):
        new = [torch.full((opt.moment_elems,), 9.0, dtype=dtype, device="cuda") for _ in range(4)]
    assert not torch.cuda.current_stream().query(), "the stream has to be behind still"
    assert not used & {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, doubled))


# ---------------------------------------------------------------- refusals

def test_binding_refuses(torch, bd):
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")
    bad = [
        lambda: bd.AdamW([z(4, 4).t()[:2]], [z(2, 4)]),                     # not contiguous
        lambda: bd.AdamW([z(4)], [z(5)]), lambda: bd.AdamW([z(4)], [z(2, 2)]),
        lambda: bd.AdamW([z(4)], [z(4), z(4)]),
        lambda: bd.AdamW([z(4, dtype=torch.float16)], [z(4)]),              # fp16 parameters
        lambda: bd.AdamW([z(4, dtype=torch.float64)], [z(4)]),
        lambda: bd.AdamW([z(4)], [z(4, dtype=torch.int32)]),
        lambda: bd.AdamW([z(4)], [z(4).cpu()]),
        lambda: bd.AdamW([z(4)], [z(4)], copies=[z(4)]),
        lambda: bd.AdamW([z(4, dtype=torch.bfloat16)], [z(4)], copies=[z(4, dtype=torch.bfloat16)]),
        lambda: bd.AdamW([z(4)], [z(4)], state_bits=16),
        lambda: bd.AdamW([z(4)], [z(4)], state_bits=[8, 8]),
        lambda: bd.AdamW([z(4)], [z(4)], m=[z(5)]), lambda: bd.AdamW([z(4)], [z(4)], state_bits=8, m=[z(4)]),
        lambda: bd.AdamW([z(4)], [z(4)], m_scale=[z(1, dtype=torch.uint8)]),
        lambda: bd.AdamW([z(4)], [z(4)], state_bits=8, v_scale=[z(2, dtype=torch.uint8)]),
        lambda: bd.GradClip([z(4, 4).t()]), lambda: bd.GradClip([z(4, dtype=torch.float64)]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    p, g = z(300), z(300)
    for f in (lambda: bd.AdamW([p, p], [g, g]), lambda: bd.AdamW([p], [p]), lambda: bd.AdamW([p], [g], m=[g]),
              lambda: bd.AdamW([p], [g], hp=bd.make_adamw_hparams(adam_eps=0.0)),
              lambda: bd.AdamW([p], [g], weight_decay=-1.0), lambda: bd.GradClip([g, g]),
              lambda: bd.AdamW([p], [g], steps_taken=-1)):
        with pytest.raises(bd.ShampooError):
            f()
    opt, clip = bd.AdamW([p], [g]), bd.GradClip([g])
    for f in (lambda: opt.step(float("nan")), lambda: opt.step(1e-3, step=-1), lambda: clip.norm(0.0),
              lambda: clip.norm(float("nan")), lambda: clip.clip(1.0, 0.0), lambda: clip.norm(1.0, float("inf")),
              lambda: opt.load_moments(z(520)[1:513], z(512))):
        with pytest.raises(bd.ShampooError):
            f()
    scalar = z(2)
    for at in ((None, scalar.data_ptr() + 2), (scalar.data_ptr() + 1, None)):  # a rate or coefficient off 4 bytes
        assert bd.load().shampoo_adamw_step(opt._ctx, 0, 1e-3, *at, opt.ws.data_ptr(), opt.ws.numel(), None) == \
            bd.SHAMPOO_EINVAL
    for f in (lambda: opt.step(1e-3, coef=z(2)), lambda: opt.step(z(1, dtype=torch.bfloat16)),
              lambda: opt.step(1e-3, coef=z(1).cpu()), lambda: opt.load_moments(z(300), z(300)),
              lambda: opt.read_moments(torch.float16), lambda: opt.read_moments(m=z(512), v=z(300)),
              lambda: opt.read_moments(torch.bfloat16, m=z(512)),
              lambda: opt.read_moments(m=z(512), v=z(512, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            f()
    ws = torch.empty(opt.ws.numel(), dtype=torch.uint8, device="cuda")
    assert bd.load().shampoo_adamw_step(opt._ctx, 0, 1e-3, None, None, ws.data_ptr(), ws.numel(),
                                        None) == bd.SHAMPOO_EINVAL  # another workspace
    assert opt.steps_taken() == 0 and not bool(p.any())


def test_buffers_that_share_memory_are_refused(torch, bd):
    n = 512
    z = lambda k=n, dtype=torch.float32: torch.zeros(k, dtype=dtype, device="cuda")
    p, g, big = z(), z(), z(2 * n + 8)
    for bits in (32, 8):
        opt, clip = bd.AdamW([p], [g], state_bits=bits), bd.GradClip([g])
        own = [opt.m[0], opt.v[0]] if bits == 32 else []
        ok = big[:n], big[n:2 * n]
        opt.read_moments(m=ok[0], v=ok[1])
        opt.load_moments(*ok)
        opt.load_moments(ok[0], ok[0])  # both are only read
        opt.load_moments(g, ok[0])
        for m, v in [(ok[0], ok[0]), (big[4:n + 4], ok[0]), (ok[1], big[n + 8:])] + \
                [(t, ok[0]) for t in own] + [(ok[0], t) for t in own]:
            with pytest.raises(bd.ShampooError):
                opt.read_moments(m=m, v=v)
        opt.read_moments(m=g, v=ok[0])  # the call has nothing else to do with gradients and parameters
        opt.load_moments(p, g)
        if bits == 8:  # codes, or scales, cut from a flat tensor
            for cut in ("m", "v", "m_scale", "v_scale"):
                flat, other = z(), z()
                k = n if len(cut) == 1 else 2
                inside = bd.AdamW([p], [g], state_bits=8, **{cut: [flat.view(torch.uint8)[100:100 + k]]})
                for f in (lambda: inside.read_moments(m=flat, v=other), lambda: inside.read_moments(m=other, v=flat),
                          lambda: inside.load_moments(flat, other), lambda: inside.load_moments(other, flat)):
                    with pytest.raises(bd.ShampooError):
                        f()
        half = big.view(torch.bfloat16)
        opt.read_moments(m=half[:n], v=half[n:2 * n])
        with pytest.raises(bd.ShampooError):
            opt.read_moments(m=half[:n], v=half[n - 8:2 * n - 8])
        for m, v in [(t, ok[0]) for t in own] + [(ok[0], t) for t in own]:
            with pytest.raises(bd.ShampooError):
                opt.load_moments(m, v)
        for s in [p[7:8]] + [t[:1] for t in own]:
            for kw in (dict(lr=s), dict(coef=s)):
                with pytest.raises(bd.ShampooError):
                    opt.step(**kw)
        opt.step(g[3:4], coef=big[:1])  # a gradient is only read: lr 0
        lib, stream = bd.load(), torch.cuda.current_stream().cuda_stream
        for at in (g.data_ptr(), g.data_ptr() + 4 * n - 4, g.data_ptr() - 4, clip.ws.data_ptr() + 8):
            assert lib.shampoo_grad_clip(clip._ctx, 1.0, 1.0, at, clip.ws.data_ptr(), clip.ws.numel(),
                                         stream) == bd.SHAMPOO_EINVAL
        assert lib.shampoo_grad_norm(clip._ctx, 1.0, 1.0, clip.ws.data_ptr() + 8, clip.ws.data_ptr(), clip.ws.numel(),
                                     stream) == bd.SHAMPOO_EINVAL
        assert opt.status() == (0, 0) and clip.norm().tolist() == [0.0, 1.0] and not bool(p.any())


# ---------------------------------------------------------------- bits

@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shapes", [[(40000,), (5001,)], [(700000,), (5001,)]])
def test_moments_are_those_of_fp32_rounded_operation_by_operation(torch, bd, bits, shapes):
    # the moments' products and sums are rounded one by one, and 8-bit roots correctly: numpy's fp32 has the same
    # bits, and with them the same codes
    f = np.float32
    opt, guard, gen = make(torch, bd, shapes, bits, torch.float32, torch.float32, None, 0)
    b1, b2 = f(opt.hp.beta1), f(opt.hp.beta2)
    for t in range(1, 6):
        for g in opt.grads:
            g.copy_(spread(torch, gen, g.numel(), 1e-2).view(g.shape))
        before = snapshot(opt)
        opt.step(1e-3)
        for i, (_, g, m0, v0) in enumerate(before):
            g, m0, v0 = g.astype(f), m0.astype(f), v0.astype(f)
            m = m0 * b1 + g * (f(1) - b1)
            v = v0 * b2 + (g * (f(1) - b2)) * g
            if bits == 32:
                assert np.array_equal(opt.m[i].cpu().numpy(), m) and np.array_equal(opt.v[i].cpu().numpy(), v)
                continue
            dm, dv, _ = oa.draws(opt.hp.seed, t, i, np.arange(len(m)))
            for x, code, scale, fmt, u in ((m, opt.m, opt.m_scale, oa.M_FORMAT, dm),
                                           (np.sqrt(v), opt.v, opt.v_scale, oa.V_FORMAT, dv)):
                e = oa.block_exponents(x, fmt)
                assert np.array_equal(scale[i].cpu().numpy().astype(int) - 127, e)
                assert np.array_equal(oa.decode(code[i].cpu().numpy(), e + 127, fmt), oa.held(x, fmt, e, u))
    guard.check()


def test_long_lists_are_dealt_out_completely(torch, bd):
    # over 16 tiles of 4096 for each block, so that tiles come from the counter, in tensors of all sizes: whole tiles,
    # short ends, other alignments, both widths; every element is stepped once, as in a list of its own
    gen = torch.Generator("cuda").manual_seed(4)
    sizes = [4096 * 700, 4096 * 300 + 17, 5, 4096, 4095, 4096 * 1500, 100001, 4096 * 64] + [4096 * 3 + 1] * 40
    P, G, M, V, S = [], [], [], [], []
    bits = [8 if i % 3 else 32 for i in range(len(sizes))]
    for i, n in enumerate(sizes):
        at = 1 if i % 5 == 4 else 0
        code = torch.uint8 if bits[i] == 8 else torch.float32
        P.append(torch.ones(n + at, device="cuda")[at:])
        G.append(torch.randn(n + at, generator=gen, device="cuda")[at:])
        M.append(torch.zeros(n + at, dtype=code, device="cuda")[at:])
        V.append(torch.zeros(n + at, dtype=code, device="cuda")[at:])
    start = [p.clone() for p in P]
    opt = bd.AdamW(P, G, state_bits=bits, m=M, v=V, weight_decay=0.0)
    for _ in range(2):
        opt.step(1e-2)
    m, v = opt.read_moments()
    assert opt.status() == (0, 0) and opt.steps_taken() == 2
    b1, b2 = opt.hp.beta1, opt.hp.beta2
    for i in range(len(sizes)):
        # Two steps of the same gradient move a parameter by 2 lr g / (|g| + eps'), eps' at most 1e-8: up to 1e-8 / |g|
        # short of 2 lr, and 1e-4 covers the roundings beside a parameter of 1.  8-bit moments are off by a code's
        # width in between: 1/8 of m (weight 0.9 * 0.1 of 0.19) and 1/16 of r (half of v), together under 0.1 of the
        # second update; and for small |g| by the formats' absolute steps in a block whose largest |g| is under 6:
        # 0.9 * 2^-9 * 2.7e-3 of m's 0.19 |g| and 1.2e-5 / 16 of r's 0.045 |g|, together under 5e-5 / |g| of the
        # second update, 3e-5 / |g| of both.
        moved = (start[i] - P[i]).double() / (2 * 0.01) * torch.sign(G[i].double())
        tol = (1e-4 if bits[i] == 32 else 0.1) + (1.1e-8 if bits[i] == 32 else 3e-5) / G[i].double().abs()
        assert bool(((moved - 1).abs() <= tol).all()), i
        if bits[i] == 32:
            g = G[i].double()
            assert bool(((opt.views(v)[i].double() / (g * g * (1 - b2 * b2)) - 1).abs() < 1e-5).all())


def test_dealt_out_tensors_have_the_bits_of_a_list_of_their_own(torch, bd):
    # each tensor of a dealt-out list against a list whose other tensors are empty (the draws go by the place in the
    # list), which is short enough for tiles in turn or for no ring at all; both widths and types, other alignments
    gen = torch.Generator("cuda").manual_seed(14)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    sizes = [4096 * 4 * sms, 4096 * 9 * sms + 17, 5, 4096, 4095, 4096 * 3 * sms, 100001] + [4096 * 3 + 1] * 20
    assert sum(-(-n // 4096) for n in sizes) >= 16 * sms  # dealt out
    spec = []
    for i, n in enumerate(sizes):
        at, bits = (1 if i % 5 == 4 else 0), (32 if i % 3 == 0 else 8)
        param = torch.bfloat16 if i % 4 == 1 else torch.float32
        spec.append((n, at, bits, torch.randn(n, generator=gen, device="cuda").to(param),
                     torch.randn(n, generator=gen, device="cuda")))

    def made(chosen):
        P, G, M, V = [], [], [], []
        for i, (n, at, bits, p, g) in enumerate(spec):
            n = n if chosen is None or i == chosen else 0
            code = torch.uint8 if bits == 8 else torch.float32
            for out, x in ((P, p), (G, g)):
                raw = torch.empty(n + at, dtype=x.dtype, device="cuda")
                raw[at:].copy_(x[:n])
                out.append(raw[at:])
            for out in (M, V):
                out.append(torch.zeros(n + at, dtype=code, device="cuda")[at:])
        opt = bd.AdamW(P, G, state_bits=[s[2] for s in spec], m=M, v=V, weight_decay=0.1)
        for _ in range(3):
            opt.step(1e-2)
        assert opt.status() == (0, 0) and opt.steps_taken() == 3
        return opt

    whole = made(None)
    for i in range(len(spec)):
        one = made(i)
        for a, b in zip((whole.params, whole.m, whole.v, whole.m_scale, whole.v_scale),
                        (one.params, one.m, one.v, one.m_scale, one.v_scale)):
            assert a[i] is None and b[i] is None or torch.equal(a[i], b[i]), i


def test_borders_of_tiles_and_shares(torch, bd):
    # a dealt-out list of one tensor against the oracle where one tile, or one share, ends and another begins: blocks
    # take shares of four tiles, a grid's width apart, and single tiles from the border on
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = 41 * sms + 3
    n = 4096 * tiles + 1003
    single = 4 * ((tiles + 1) // (4 * sms) - 1) * sms
    P = [torch.full((n,), 1.0, dtype=torch.bfloat16, device="cuda")]
    G = [torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(21))]
    opt = bd.AdamW(P, G, state_bits=8, weight_decay=0.1)
    opt.step(1e-2)
    assert opt.status() == (0, 0)
    ends = [1, sms, 4 * sms, 5 * sms, single - sms, single - 1, single, single + 1, single + sms, tiles - 1, tiles]
    check_slices(torch, opt, [(0, 512)] + [(4096 * t - 256, min(4096 * t + 256, n)) for t in ends] + [(n - n % 256, n)])


def test_counter_goes_on_from_a_late_step(torch, bd):
    p, g = torch.ones(1, device="cuda"), torch.ones(1, device="cuda")
    opt = bd.AdamW([p], [g], steps_taken=10 ** 6)
    for _ in range(5):
        opt.step(0.0)
    assert opt.steps_taken() == 10 ** 6 + 5


def test_waits_for_tiles_are_bounded(torch, bd):
    # the loads of one step are withheld: its waits run out, the launch ends and says so, and the next step is whole
    p, g = torch.ones(4096 * 200 + 5, device="cuda"), torch.ones(4096 * 200 + 5, device="cuda")
    opt = bd.AdamW([p], [g], state_bits=8, weight_decay=0.0)
    assert bd.load().shampoo_debug_inject_timeout() == 0
    opt.step(1e-2)
    assert opt.status() == (bd.SHAMPOO_ETIMEOUT, 2)
    for t in (p, g):
        t.fill_(1.0)
    for t in opt.m + opt.v + opt.m_scale + opt.v_scale:
        t.zero_()
    opt.step(1e-2, step=1)
    assert opt.status() == (0, 0) and opt.steps_taken() == 1
    assert bool(((p - 0.99).abs() <= 1e-6).all())


def test_steps_without_loads_to_withhold_leave_the_fault_armed(torch, bd):
    # the hook is for the next step that fetches tiles ahead: not one of few tiles, nor one whose tiles bulk copies
    # cannot reach
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    one = lambda n, off=0: torch.ones(n + off, device="cuda")[off:]
    short = bd.AdamW([one(4096 * sms)], [one(4096 * sms)])
    odd = bd.AdamW([one(4096 * 2 * sms, 1)], [one(4096 * 2 * sms)])
    small = bd.AdamW([one(4095) for _ in range(2 * sms)], [one(4095) for _ in range(2 * sms)])
    long = bd.AdamW([one(4096 * (sms + 1))], [one(4096 * (sms + 1))])
    assert bd.load().shampoo_debug_inject_timeout() == 0
    for opt in (short, odd, small):
        opt.step(1e-2)
        assert opt.status() == (0, 0)
        assert all(bool(((p - 0.99).abs() <= 1e-6).all()) for p in opt.params)
    long.step(1e-2)
    assert long.status() == (bd.SHAMPOO_ETIMEOUT, 2)
    long.step(1e-2)
    assert long.status() == (0, 0)


@pytest.mark.parametrize("bits", [32, 8])
def test_betas_of_zero(torch, bd, bits):
    hp = bd.make_adamw_hparams(beta1=0.0, beta2=0.0, seed=1)
    opt, guard, gen = make(torch, bd, [(5000,), (3,)], bits, torch.float32, torch.float32, None, 0, hp=hp)
    for t in range(1, 4):
        for g in opt.grads:
            g.copy_(torch.randn(g.shape, generator=gen))
        before = snapshot(opt)
        opt.step(1e-2)
        check_step(torch, opt, before, t, 1e-2)
    guard.check()


def test_parameters_of_a_module_on_a_stream_of_ones_own(torch, bd):
    # nn.Parameters with their .grad, made and stepped inside a stream context, moments in and out captured
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        net = torch.nn.Sequential(torch.nn.Linear(70, 90), torch.nn.LayerNorm(90)).cuda()
        net(torch.randn(8, 70, device="cuda")).square().sum().backward()
        params = list(net.parameters())
        opt = bd.AdamW(params, [p.grad for p in params], state_bits=[8, 32, 8, 32])
        clip = bd.GradClip([p.grad for p in params])
        old = [p.detach().clone() for p in params]
        opt.step(1e-2, coef=clip.norm(1.0)[1:])
        assert opt.status() == (0, 0)
        assert all(not torch.equal(a, p) for a, p in zip(old, params) if bool(p.grad.any()))
        m, v = opt.read_moments()
        copy = [t.clone() for t in opt.m + opt.v]
        graph = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            opt.load_moments(m, v)
            out = opt.read_moments(torch.bfloat16)
        for t in opt.m + opt.v:
            t.zero_()
        graph.replay()
        s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copy[1::2], (opt.m + opt.v)[1::2]))
    assert torch.equal(out[0], m.bfloat16()) and torch.equal(out[1], v.bfloat16())


def test_list_without_elements(torch, bd):
    e = lambda: torch.zeros(0, device="cuda")
    for bits in (32, 8):
        opt = bd.AdamW([e(), e()], [e(), e()], state_bits=bits)
        assert opt.moment_elems == 0
        for _ in range(3):
            opt.step(1e-3)
        opt.load_moments(e(), e())
        assert [t.numel() for t in opt.read_moments()] == [0, 0]
        assert opt.status() == (0, 0) and opt.steps_taken() == 3


def test_thousands_of_small_tensors(torch, bd):
    # the search for a tile's tensor goes 32 ways over several levels
    rng = np.random.default_rng(6)
    sizes = rng.integers(0, 600, 5000).tolist()
    total = sum(sizes)
    gen = torch.Generator("cuda").manual_seed(8)
    flat = {k: torch.randn(total, generator=gen, device="cuda") for k in "pg"}
    start = flat["p"].clone()
    ends = np.cumsum([0] + sizes)
    cut = lambda x: [x[a:b] for a, b in zip(ends[:-1], ends[1:])]
    opt = bd.AdamW(cut(flat["p"]), cut(flat["g"]), state_bits=[8 if i % 2 else 32 for i in range(5000)])
    clip = bd.GradClip(cut(flat["g"]))
    opt.step(0.5)
    # eps' beside |g|, and a dozen roundings of the update and one of the parameter
    g = flat["g"].double()
    want = start.double() - 0.5 * g / (g.abs() + float(np.float32(1e-8)))
    assert bool(((flat["p"].double() - want).abs() <= 0.5 * 16 * H + H * want.abs() * 1.01 + 1e-15).all())
    m, _ = opt.read_moments()
    for i in (0, 1, 31, 32, 33, 1023, 1024, 1025, 4998, 4999):
        if sizes[i]:
            x = f64(opt.views(m)[i]) / (0.1 * f64(opt.grads[i]))
            assert np.all(np.abs(x[np.abs(f64(opt.grads[i])) > 0.05] - 1) < (1e-6 if i % 2 == 0 else 0.13))
    n = math.sqrt(float((g * g).sum()))
    assert abs(clip.norm()[0].item() - n) <= 1.01 * H * n
