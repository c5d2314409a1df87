"""GPU tests of the global gradient norm and clipping, alone and together with
the Shampoo and AdamW steps.

The squares and their sum are formed in fp64, so norm and coef are the exact
ones rounded to fp32, half a step (2^-24) off and a little more for the fp64
sums; a clipped gradient has one more rounding of coef g to fp32, and one to
its type.
"""

import math

import numpy as np
import pytest

from matrix_inverse_roots_stack_b200 import workloads
from oracle import adamw as oa, step as ostep
from tests.gpu_util import cuda_or_skip, rel

pytestmark = pytest.mark.gpu

H = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    return cuda_or_skip()


@pytest.fixture(scope="module")
def bd():
    from matrix_inverse_roots_stack_b200 import binding
    return binding


def grads_of(torch, sizes, dtype, offset, seed=0, std=1e-2):
    gen = torch.Generator().manual_seed(seed)
    out = []
    for n in sizes:
        raw = torch.full((n + offset + 64,), 3.0, dtype=dtype, device="cuda")
        g = raw[offset:offset + n]
        g.copy_(torch.randn(n, generator=gen) * std)
        out.append(g)
    return out


SIZES = [[1], [0, 7, 0], [8191, 8192, 8193], [16383, 16384, 16385], [1, 255, 256, 257, 100003], [3_000_001]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("offset", [0, 1, 4, 8])
def test_norm_and_clip(torch, bd, sizes, dtype, offset):
    dtype = getattr(torch, dtype)
    grads = grads_of(torch, sizes, dtype, offset)
    clip = bd.GradClip(grads)
    ref = [g.double().cpu().numpy() for g in grads]
    n0, _ = oa.norm_and_coef(ref, math.inf, 1.0)
    for max_norm, inv_scale in ((math.inf, 1.0), (float(np.float32(n0 / 2)), 1.0), (float(np.float32(n0 * 2)), 1.0),
                                (float(np.float32(n0 * 2)), 4.0), (math.inf, 2.0 ** -10), (float(np.float32(1e-30)), 1.0)):
        n, c = oa.norm_and_coef(ref, max_norm, inv_scale)
        norm, coef = clip.norm(max_norm, inv_scale).tolist()
        assert abs(norm - n) <= 1.01 * H * n and abs(coef - c) <= 1.01 * H * c
        again = clip.norm(max_norm, inv_scale).tolist()
        assert (norm, coef) == tuple(again) and clip.status() == (0, 0)
    assert all(np.array_equal(g.double().cpu().numpy(), r) for g, r in zip(grads, ref))  # only read
    n, c = oa.norm_and_coef(ref, float(np.float32(n0 / 2)), 1.0)
    got = clip.clip(float(np.float32(n0 / 2))).tolist()
    assert abs(got[1] - c) <= 1.01 * H * c
    info = torch.finfo(dtype)
    for g, r in zip(grads, ref):
        x = g.double().cpu().numpy()
        want = got[1] * r
        # one rounding to fp32 (none beside the type's own for fp32), one to the type
        tol = np.abs(want) * (info.eps / 2 + (H if dtype != torch.float32 else 0)) * 1.01 + info.tiny * info.eps / 2
        assert np.all(np.abs(x - want) <= tol)
    for g in grads:  # what lies around them is as it was
        raw = g._base if g._base is not None else g
        if g.numel():
            assert bool((raw[:offset] == 3).all()) and bool((raw[offset + g.numel():] == 3).all())


@pytest.mark.parametrize("chunks_an_sm", [1, 3, 5, 7, 10, 14, 20, 30, 50, 100, 170])
def test_long_lists(torch, bd, chunks_an_sm):
    # chunks of 32 KB, from one an SM to more than 16 for each block that the device holds (two to eight an SM): one
    # share a block, shares from the counter, of one chunk and of several, the last group short.  All types and odd
    # ends, some tensors off 16 bytes.  Equal bits of every share's sum, which the workspace keeps, whatever else the
    # device is doing
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = sms * chunks_an_sm * 8192 // 4  # fp32 elements of a quarter of the list
    gen = torch.Generator("cuda").manual_seed(chunks_an_sm)
    grads = []
    for dtype, size, offset in ((torch.float32, n + 5, 0), (torch.bfloat16, 2 * n - 3, 0), (torch.float16, 2 * n + 1, 0),
                                (torch.bfloat16, n, 1), (torch.float32, n // 2 + 77, 1)):
        raw = torch.empty(size + offset, dtype=dtype, device="cuda")
        raw.normal_(generator=gen)
        grads.append(raw[offset:])
    want = math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))
    clip = bd.GradClip(grads)
    norm = clip.norm(want / 2)[0].item()
    assert abs(norm - want) <= 1.01 * H * want and clip.status() == (0, 0)
    kept, out = clip.ws.clone(), clip.out.clone()
    side, busy = torch.cuda.Stream(), torch.empty(1 << 24, device="cuda")
    torch.cuda.synchronize()
    for k in range(20):
        with torch.cuda.stream(side):
            for _ in range(k % 4):
                busy.normal_()
        clip.norm(want / 2)
        assert torch.equal(clip.ws, kept) and torch.equal(clip.out, out)
    torch.cuda.synchronize()
    if chunks_an_sm in (3, 20):
        before = [g.clone() for g in grads]
        coef = clip.clip(want / 2)[1]
        for g, b in zip(grads, before):  # the product in fp32, rounded to the type
            assert torch.equal(g, (b.float() * coef).to(g.dtype))


@pytest.mark.parametrize("value", [1e-38, 1e-30, 1e25, 3e38])
def test_extreme_values(torch, bd, value):
    g = torch.full((5000,), value, device="cuda")
    clip = bd.GradClip([g])
    x = float(np.float32(value))
    n = math.sqrt(5000) * x
    norm, coef = clip.norm(1.0).tolist()
    assert clip.status() == (0, 0)
    assert (norm == math.inf if n > 3.4e38 else abs(norm - n) <= 1.01 * H * n)
    c = min(1.0, 1.0 / n)
    assert abs(coef - c) <= 1.01 * H * c + 2.0 ** -150  # coef may lie below fp32's normal range
    clip.clip(1e3)
    want = x * min(1.0, 1e3 / n)
    assert abs(g[17].item() - want) <= want * 3 * H + x * 2.0 ** -150


def test_zero_and_empty(torch, bd):
    g = torch.zeros(300, device="cuda")
    clip = bd.GradClip([g, torch.zeros(0, device="cuda")])
    assert clip.norm(1.0, 0.5).tolist() == [0.0, 0.5] and clip.clip(1.0).tolist() == [0.0, 1.0]
    empty = bd.GradClip([torch.zeros(0, device="cuda")])
    assert empty.clip(1.0).tolist() == [0.0, 1.0] and empty.status() == (0, 0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_non_finite(torch, bd, bad, dtype):
    grads = grads_of(torch, [70000, 100], getattr(torch, dtype), 1)
    clip = bd.GradClip(grads)
    grads[0][69999] = bad
    norm, coef = clip.norm(1.0).tolist()
    assert not math.isfinite(norm) and math.isnan(coef) and clip.status() == (bd.SHAMPOO_ENONFINITE, 1)
    assert not bool(torch.isfinite(grads[0][69999]))
    clip.clip(1.0)
    assert clip.status()[0] == bd.SHAMPOO_ENONFINITE
    assert not any(bool(g.any()) for g in grads)
    assert clip.norm(1.0).tolist() == [0.0, 1.0] and clip.status() == (0, 0)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_non_finite_at_any_place_of_a_whole_chunk(torch, bd, dtype):
    g = torch.ones(16384 * 3, dtype=getattr(torch, dtype), device="cuda")
    clip = bd.GradClip([g])
    for at in (0, 1, 2, 7, 255, 256, 8190, 8191, 8192, 16383, 16384, 3 * 16384 - 2, 3 * 16384 - 1):
        for bad in (float("nan"), float("inf"), -float("inf")):
            g[at] = bad
            norm, coef = clip.norm(1.0).tolist()
            assert not math.isfinite(norm) and math.isnan(coef) and clip.status()[0] == bd.SHAMPOO_ENONFINITE
        g[at] = 1.0
    n = math.sqrt(16384 * 3)
    assert clip.norm()[0].item() == np.float32(n) and clip.status() == (0, 0)


@pytest.mark.parametrize("values", [(1e-39, 9.2e-41), (1e-39, 0.0), (0.0, 1e-39), (3e38, 1.0), (1.0, 3e38),
                                    (-1e-20, 1e-20), (0.0, 0.0), (-2.5, 1e-30)])
def test_bf16_values_of_any_size(torch, bd, values):
    # even and odd elements are converted differently: subnormal, zero and near the largest, in both places
    g = torch.tensor(values, device="cuda").to(torch.bfloat16).repeat(8192)
    clip = bd.GradClip([g])
    n = math.sqrt(float(g.double().square().sum()))
    norm = clip.norm(1e30)[0].item()
    assert clip.status() == (0, 0)
    assert norm == math.inf if n > 3.4028235e38 else abs(norm - n) <= 1.01 * H * n + 2.0 ** -150


def test_captured_clip_replays(torch, bd):
    grads = grads_of(torch, [100003, 77], torch.float32, 0)
    twin = [g.clone() for g in grads]
    clip, ref = bd.GradClip(grads), bd.GradClip(twin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clip.clip(0.5)
    for k in range(3):
        for a, b in zip(grads, twin):
            a.normal_(generator=torch.Generator("cuda").manual_seed(k))
            b.copy_(a)
        graph.replay()
        ref.clip(0.5)
        assert all(torch.equal(a, b) for a, b in zip(grads, twin)) and torch.equal(clip.out, ref.out)


def test_shampoo_and_adamw_share_one_clipped_step(torch, bd):
    # a model's step: all gradients clipped by one norm, matrices by Shampoo, the embedding (8-bit moments), norm
    # weights and biases by AdamW; against the oracles on the clipped gradients, and a skipped step in between
    rng = np.random.default_rng(11)
    mats = [(256, 384), (128, 200)]
    rest = [(1000, 64), (384,), (7,)]
    P = [torch.from_numpy((0.02 * rng.standard_normal(s)).astype(np.float32)).cuda() for s in mats + rest]
    G = [torch.zeros_like(p) for p in P]
    hp = ostep.HParams(block_size=128, ndb_iters1=14, ndb_iters2=14, eps=1e-4)
    v0 = workloads.pi_start_vectors(128, 32, seed=0)
    shampoo = bd.Shampoo(P[:2], G[:2], v0=torch.from_numpy(v0).cuda(),
                         hp=bd.make_hparams(block_size=128, ndb_iters1=14, ndb_iters2=14, eps=1e-4))
    adamw = bd.AdamW(P[2:], G[2:], state_bits=[8, 32, 32], weight_decay=[0.1, 0.0, 0.0])
    clip_all, clip_mats = bd.GradClip(G), bd.GradClip(G[:2])
    g0 = [rng.standard_normal(s).astype(np.float32) for s in mats + rest]
    for g, x in zip(G, g0):
        g.copy_(torch.from_numpy(x))
    start = [p.double().cpu().numpy() for p in P]
    n, c = oa.norm_and_coef(g0, 1.0, 1.0)

    clip_all.clip(1.0)
    shampoo.step()
    adamw.step(1e-2)
    assert shampoo.status()[0] == 0 and adamw.status()[0] == 0 and clip_all.status()[0] == 0
    b = [float(np.float32(x)) for x in (0.9, 0.999, 1e-8, 1e-2)]
    for i in range(2, 5):
        wd = float(np.float32(0.1)) if i == 2 else 0.0
        want, _, _ = oa.step(start[i], c * g0[i], 0.0, 0.0, 1, *b, wd)
        # the update is lr g / (|g| + eps): about 30 roundings of it, and one of the parameter
        d = np.abs(P[i].double().cpu().numpy() - want)
        assert np.all(d <= 0.01 * 30 * H + np.abs(want) * 1.01 * H)
    lam = shampoo.lam.cpu().numpy().astype(np.float64)
    import dataclasses
    hp = dataclasses.replace(hp, **{f: float(np.float32(getattr(hp, f))) for f in (
        "beta", "eps", "init_scale", "beta1", "beta2", "adam_eps", "lr")})
    new, _, _ = ostep.shampoo_step(start[:2], [c * g.astype(np.float64) for g in g0[:2]],
                                   ostep.init_state(mats, hp), hp, v0.astype(np.float64), lam_override=lam)
    for i in range(2):
        assert rel(P[i].double().cpu().numpy() - start[i], new[i] - start[i]) < 5e-3

    # a step with a non-finite gradient: clipping zeroes Shampoo's gradients, AdamW is told by coef
    kept = [p.clone() for p in P]
    for g, x in zip(G, g0):
        g.copy_(torch.from_numpy(x))
    G[3][5] = float("inf")
    coef = clip_all.norm(1.0)[1:]
    adamw.step(1e-2, coef=coef)
    clip_all.clip(1.0)
    shampoo.step()
    assert shampoo.status()[0] == 0 and adamw.steps_taken() == 1
    assert clip_all.status()[0] == bd.SHAMPOO_ENONFINITE
    assert all(torch.equal(a, p) for a, p in zip(kept, P))
    assert clip_mats.norm().tolist() == [0.0, 1.0]
