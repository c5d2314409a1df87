"""Host-side checks of the operators over a list of tensors (no GPU): what
the C entry points refuse, and the oracle's 8-bit formats and draws."""

import ctypes

import numpy as np
import pytest

from matrix_inverse_roots_stack_b200 import binding as bd
from oracle import adamw as oa


@pytest.fixture(scope="module")
def lib():
    from matrix_inverse_roots_stack_b200 import build
    build.build()
    return bd.load()


# ---------------------------------------------------------------- gradient lists

def grads_init(lib, rows):
    arr = (bd.ShampooGrad * max(len(rows), 1))(*[bd.ShampooGrad(*r) for r in rows])
    ctx, n = ctypes.c_void_p(), ctypes.c_size_t()
    rc = lib.shampoo_grads_init(ctypes.byref(ctx), arr, len(rows), ctypes.byref(n))
    return rc, ctx, n.value


@pytest.mark.parametrize("rows,ok", [
    ([(100, 0x1000, bd.DTYPE_F32)], True),
    ([(100, 0x1002, bd.DTYPE_BF16), (100, 0x10ca, bd.DTYPE_F16)], True),   # adjacent
    ([(0, None, bd.DTYPE_F32)], True),
    ([(100, 0x1002, bd.DTYPE_F32)], False),                                # not even its type's alignment
    ([(100, 0x1001, bd.DTYPE_BF16)], False),
    ([(100, None, bd.DTYPE_F32)], False),
    ([(-1, 0x1000, bd.DTYPE_F32)], False),
    ([((1 << 40) + 1, 0x1000, bd.DTYPE_F32)], False),
    ([(100, 0x1000, 3)], False),
    ([(100, 0x1000, bd.DTYPE_F32), (100, 0x1000, bd.DTYPE_F32)], False),   # the same tensor twice
    ([(100, 0x1000, bd.DTYPE_F32), (100, 0x118c, bd.DTYPE_F32)], False),   # the last element shared
    ([], False),
])
def test_gradient_list(lib, rows, ok):
    rc, ctx, nbytes = grads_init(lib, rows)
    assert rc == (bd.SHAMPOO_OK if ok else bd.SHAMPOO_EINVAL)
    assert (nbytes > 0) == ok and bool(ctx.value) == ok
    lib.shampoo_grads_destroy(ctx)


def test_gradient_calls_validate_before_device_work(lib):
    rc, ctx, need = grads_init(lib, [(100, 0x1000, bd.DTYPE_F32)])
    assert rc == 0
    ws, out = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x2000)
    assert lib.shampoo_grads_bind(None, ws, need, None) == bd.SHAMPOO_EINVAL
    assert lib.shampoo_grads_bind(ctx, None, need, None) == bd.SHAMPOO_EWORKSPACE
    assert lib.shampoo_grads_bind(ctx, ws, need - 1, None) == bd.SHAMPOO_EWORKSPACE
    assert lib.shampoo_grads_bind(ctx, ctypes.c_void_p(0x100010), need, None) == bd.SHAMPOO_EWORKSPACE
    for fn in (lib.shampoo_grad_norm, lib.shampoo_grad_clip):
        assert fn(None, 1.0, 1.0, out, ws, need, None) == bd.SHAMPOO_EINVAL
        assert fn(ctx, 1.0, 1.0, None, ws, need, None) == bd.SHAMPOO_EINVAL
        assert fn(ctx, 1.0, 1.0, out, None, need, None) == bd.SHAMPOO_EWORKSPACE
        assert fn(ctx, 1.0, 1.0, out, ws, need - 1, None) == bd.SHAMPOO_EWORKSPACE
        assert fn(ctx, 1.0, 1.0, out, ws, need, None) == bd.SHAMPOO_EINVAL  # not bound
        for max_norm, inv_scale in ((0.0, 1.0), (-1.0, 1.0), (float("nan"), 1.0), (1.0, 0.0), (1.0, -1.0),
                                    (1.0, float("inf")), (1.0, float("nan"))):
            assert fn(ctx, max_norm, inv_scale, out, ws, need, None) == bd.SHAMPOO_EINVAL
        assert fn(ctx, 1.0, 1.0, ctypes.c_void_p(0x2002), None, need, None) == bd.SHAMPOO_EINVAL  # out off 4 bytes
    lib.shampoo_grads_destroy(ctx)
    lib.shampoo_grads_destroy(None)


# ---------------------------------------------------------------- AdamW lists

def tensor(base=0x10000, n=1000, **changes):
    t = dict(n=n, param=base, grad=base + 0x10000, copy=None, m=base + 0x20000, v=base + 0x30000, m_scale=None,
             v_scale=None, param_dtype=bd.DTYPE_F32, grad_dtype=bd.DTYPE_F32, copy_dtype=bd.DTYPE_F32, state_bits=32,
             lr_scale=1.0, weight_decay=0.1)
    if changes.get("state_bits") == 8:
        t.update(m_scale=base + 0x40000, v_scale=base + 0x41000)
    t.update(changes)
    return bd.AdamwTensor(**t)


def adamw_init(lib, tensors, **hp):
    arr = (bd.AdamwTensor * max(len(tensors), 1))(*tensors)
    ctx, n, elems = ctypes.c_void_p(), ctypes.c_size_t(), ctypes.c_int64(-1)
    h = bd.make_adamw_hparams(**hp)
    rc = lib.shampoo_adamw_init(ctypes.byref(ctx), arr, len(tensors), ctypes.byref(h), ctypes.byref(n),
                                ctypes.byref(elems))
    return rc, ctx, n.value, elems.value


@pytest.mark.parametrize("changes", [
    {}, {"state_bits": 8}, {"n": 0}, {"n": 0, "param": None, "grad": None, "m": None, "v": None},
    {"param_dtype": bd.DTYPE_BF16}, {"grad_dtype": bd.DTYPE_F16}, {"copy": 0x70000, "copy_dtype": bd.DTYPE_BF16},
    {"lr_scale": 0.0}, {"weight_decay": 0.0}, {"param": 0x10004},
    {"state_bits": 8, "m": 0x30001, "v": 0x40003, "m_scale": 0x50007}])
def test_adamw_list_accepts(lib, changes):
    rc, ctx, nbytes, elems = adamw_init(lib, [tensor(**changes)])
    assert rc == bd.SHAMPOO_OK and nbytes > 0
    assert elems == -(-changes.get("n", 1000) // bd.QBLOCK) * bd.QBLOCK
    lib.shampoo_adamw_destroy(ctx)


@pytest.mark.parametrize("changes", [
    {"n": -1}, {"n": (1 << 40) + 1}, {"param": None}, {"grad": None}, {"m": None}, {"v": None},
    {"param_dtype": bd.DTYPE_F16}, {"param_dtype": 5}, {"grad_dtype": -1}, {"state_bits": 16}, {"state_bits": 4},
    {"state_bits": 8, "m_scale": None}, {"state_bits": 8, "v_scale": None},
    {"copy": 0x70000, "copy_dtype": bd.DTYPE_F32},
    {"copy": 0x70000, "copy_dtype": bd.DTYPE_BF16, "param_dtype": bd.DTYPE_BF16},
    {"copy": 0x70001, "copy_dtype": bd.DTYPE_BF16}, {"param": 0x10002}, {"grad": 0x20001}, {"m": 0x30002},
    {"lr_scale": -1.0}, {"lr_scale": float("nan")}, {"weight_decay": -0.1}, {"weight_decay": float("inf")},
    {"grad": 0x10000}, {"m": 0x10000}, {"v": 0x30000 + 3996}, {"copy": 0x10000, "copy_dtype": bd.DTYPE_BF16},
    {"state_bits": 8, "v_scale": 0x50003}])  # four blocks of scales at 0x50000
def test_adamw_list_refuses(lib, changes):
    rc, ctx, nbytes, _ = adamw_init(lib, [tensor(**changes)])
    assert rc == bd.SHAMPOO_EINVAL and not ctx.value


def test_adamw_list_refuses_shared_parameters(lib):
    assert adamw_init(lib, [])[0] == bd.SHAMPOO_EINVAL
    assert adamw_init(lib, [tensor(), tensor()])[0] == bd.SHAMPOO_EINVAL
    two = [tensor(), tensor(0x80000)]
    rc, ctx, _, elems = adamw_init(lib, two)
    assert rc == bd.SHAMPOO_OK and elems == 2048
    lib.shampoo_adamw_destroy(ctx)
    # a gradient may be shared (it is only read), but is no other's parameter
    rc, ctx, _, _ = adamw_init(lib, [tensor(), tensor(0x80000, grad=0x20000)])
    assert rc == bd.SHAMPOO_OK
    lib.shampoo_adamw_destroy(ctx)
    assert adamw_init(lib, [tensor(), tensor(0x80000, grad=0x10000)])[0] == bd.SHAMPOO_EINVAL


@pytest.mark.parametrize("hp", [{"beta1": 1.0}, {"beta1": -0.1}, {"beta2": 1.0}, {"beta2": float("nan")},
                                {"adam_eps": 0.0}, {"adam_eps": 1e-40}, {"adam_eps": float("inf")}])
def test_adamw_hparams(lib, hp):
    assert adamw_init(lib, [tensor()], **hp)[0] == bd.SHAMPOO_EINVAL


def test_adamw_calls_validate_before_device_work(lib):
    rc, ctx, need, _ = adamw_init(lib, [tensor()])
    assert rc == 0
    ws, p = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x2000)
    assert lib.shampoo_adamw_bind(None, 0, ws, need, None) == bd.SHAMPOO_EINVAL
    assert lib.shampoo_adamw_bind(ctx, -1, ws, need, None) == bd.SHAMPOO_EINVAL
    assert lib.shampoo_adamw_bind(ctx, 0, None, need, None) == bd.SHAMPOO_EWORKSPACE
    assert lib.shampoo_adamw_bind(ctx, 0, ws, need - 1, None) == bd.SHAMPOO_EWORKSPACE
    assert lib.shampoo_adamw_bind(ctx, 0, ctypes.c_void_p(0x100080), need, None) == bd.SHAMPOO_EWORKSPACE
    calls = [lambda w, n: lib.shampoo_adamw_step(ctx, 0, 1e-3, None, None, w, n, None),
             lambda w, n: lib.shampoo_adamw_load_moments(ctx, p, p, w, n, None),
             lambda w, n: lib.shampoo_adamw_read_moments(ctx, p, p, bd.DTYPE_F32, w, n, None),
             lambda w, n: lib.shampoo_adamw_steps_taken(ctx, w, n, None, ctypes.byref(ctypes.c_int()))]
    for call in calls:
        assert call(None, need) == bd.SHAMPOO_EWORKSPACE
        assert call(ws, need - 1) == bd.SHAMPOO_EWORKSPACE
        assert call(ws, need) == bd.SHAMPOO_EINVAL  # not bound
    assert lib.shampoo_adamw_step(None, 0, 1e-3, None, None, ws, need, None) == bd.SHAMPOO_EINVAL
    lib.shampoo_adamw_destroy(ctx)
    lib.shampoo_adamw_destroy(None)


def test_header_constants(lib):
    text = open(lib._name.replace("matrix_inverse_roots_stack_b200/libdash_b200.so", "include/dash_b200.h")).read()
    for name, value in (("DTYPE_F32", bd.DTYPE_F32), ("DTYPE_BF16", bd.DTYPE_BF16), ("DTYPE_F16", bd.DTYPE_F16),
                        ("QBLOCK", bd.QBLOCK)):
        assert f"#define SHAMPOO_{name} {value}" in text
    assert oa.BLOCK == bd.QBLOCK


@pytest.mark.parametrize("make", [
    lambda t: bd.GradClip([]), lambda t: bd.GradClip([t.zeros(4)]),
    lambda t: bd.AdamW([], []), lambda t: bd.AdamW([t.zeros(4)], [t.zeros(4)])])
def test_binding_refuses_lists_without_cuda_tensors(lib, make):
    with pytest.raises(ValueError):
        make(pytest.importorskip("torch"))


def test_workspace_shares_no_memory_with_the_list(lib):
    # two tensors with a hole between them; a workspace that reaches into either, or lies around one, is refused
    # before anything is uploaded, one in the hole or behind goes on to the device
    gpu = pytest.importorskip("torch").cuda.is_available()
    rc, grads, need = grads_init(lib, [(100, 0x100000, bd.DTYPE_F32), (100, 0x300000, bd.DTYPE_F32)])
    rc2, adamw, need2, _ = adamw_init(lib, [tensor(0x100000), tensor(0x300000, grad=0x110000)])
    assert rc == 0 and rc2 == 0
    for bind, ctx, n in ((lambda *a: lib.shampoo_grads_bind(*a, None), grads, need),
                         (lambda c, *a: lib.shampoo_adamw_bind(c, 0, *a, None), adamw, need2)):
        low = -(-n // 256) * 256
        for at, ok in ((0x100000, False), (0x300000, False), (0x300100, False), (0x300000 - low, True),
                       (0x300000 - low + 256, n <= low - 256), (0x100000 - low, True), (0x100000 - 256, n <= 256),
                       (0x800000, True), (0x200000, True)):
            if not (ok and gpu):  # no made-up address goes to a device
                assert (bind(ctx, ctypes.c_void_p(at), n) != bd.SHAMPOO_EINVAL) == ok, hex(at)
    # arrays of which others are read only
    for at in (0x110000, 0x120000, 0x130f00, 0x320000):
        assert lib.shampoo_adamw_bind(adamw, 0, ctypes.c_void_p(at), need2, None) == bd.SHAMPOO_EINVAL
    lib.shampoo_grads_destroy(grads)
    lib.shampoo_adamw_destroy(adamw)


# ---------------------------------------------------------------- the oracle's formats

@pytest.mark.parametrize("fmt", [oa.M_FORMAT, oa.V_FORMAT])
def test_every_code_is_held_exactly(fmt):
    bits = 128 if fmt is oa.M_FORMAT else 256
    codes = np.arange(bits - (fmt is oa.M_FORMAT))  # 0x7f is not a number of e4m3
    x = oa.decode(codes, np.full(1, 127), fmt)
    assert np.all(np.diff(x) > 0) and x[0] == 0 and x[-1] == fmt[2]
    assert oa.block_exponents(x, fmt) == [0]
    for u in (None, np.zeros(len(x), int), np.full(len(x), 65535)):
        assert np.array_equal(oa.held(x, fmt, [0], u), x)
    assert oa.block_exponents(x * 2.0 ** -30, fmt) == [-30]
    assert oa.block_exponents([fmt[2] * (1 + 2.0 ** -30)], fmt) == [1]


def test_e4m3_is_torchs():
    torch = pytest.importorskip("torch")
    codes = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(oa.decode(codes, np.full(1, 127), oa.M_FORMAT), ref)


def test_draws_are_uniform_and_independent():
    # each statistic is a mean of n products of independent unit-variance
    # variables, about N(0, 1/n); 6 sigma over the few hundred looks below
    n = 1 << 18
    i = np.arange(n) + (1 << 32) - n // 2
    prev = None
    for t in range(1, 9):
        d = [(x.astype(np.float64) + 0.5) / 65536 - 0.5 for x in oa.draws(12345678901, t, 3, i)]
        d = [x * np.sqrt(12) for x in d]
        looks = [x for x in d] + [d[0] * d[1], d[0] * d[2], d[1] * d[2]]
        for lag in (1, 2, 8, 32, 256, 2048):
            looks += [x[:-lag] * x[lag:] for x in d]
        if prev is not None:
            looks += [a * b for a, b in zip(d, prev)]
        prev = d
        for x in looks:
            assert abs(x.mean()) * np.sqrt(len(x)) < 6
    assert not np.array_equal(oa.draws(1, 1, 0, i)[0], oa.draws(1, 1, 1, i)[0])
    assert not np.array_equal(oa.draws(1, 1, 0, i)[0], oa.draws(1 + (1 << 32), 1, 0, i)[0])


# ---------------------------------------------------------------- the binding's streams

class FakeMemory:
    """What read_moments looks at in a tensor, and the stream that was current
    when its memory was handed out."""

    def __init__(self, n, dtype, on):
        self.n, self.dtype, self.on, self.recorded = n, dtype, on, []

    numel = lambda self: self.n
    is_contiguous = lambda self: True
    get_device = lambda self: 0
    data_ptr = lambda self: 0x1000

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.mark.parametrize("given", ["", "m", "v"])
def test_outputs_come_from_the_memory_of_the_stream_that_writes_them(monkeypatch, given):
    torch = pytest.importorskip("torch")
    import contextlib
    import types
    device = torch.device("cuda", 0)
    ours, side = (types.SimpleNamespace(device=device, cuda_stream=h) for h in (7, 8))
    current = [ours]

    @contextlib.contextmanager
    def stream(s):
        current.append(current[-1] if s is None else s)
        yield
        current.pop()

    fake = types.SimpleNamespace(stream=stream, current_stream=lambda device=None: current[-1])
    monkeypatch.setattr(torch, "cuda", fake)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: FakeMemory(n, dtype, current[-1]))

    def read(ctx, m, v, dtype, ws, ws_bytes, handle):
        handles.append(handle)
        return 0

    opt = bd.AdamW.__new__(bd.AdamW)
    opt.device, opt._index, opt.moment_elems = device, 0, 512
    opt._cuda, opt._device, opt._current = fake, lambda: 0, lambda index: current[-1].cuda_stream
    opt._ctx, opt._ws_at, opt._ws_bytes, opt._held, opt._streams = None, 0, 0, [], {7, 8}
    opt._dtypes, opt._read = {torch.float32: bd.DTYPE_F32, torch.bfloat16: bd.DTYPE_BF16}, read
    for s in (None, side):
        handles = []
        passed = {k: FakeMemory(512, torch.float32, ours) for k in given}
        out = dict(zip("mv", opt.read_moments(stream=s, **passed)))
        assert handles == [7 if s is None else 8] and current == [ours]
        for k, t in out.items():
            if k in passed:
                assert t is passed[k] and (s is None or side in t.recorded)
            else:  # another stream's memory would still be in that one's use
                assert t.on is (ours if s is None else side)
                assert s is None or ours in t.recorded


def fake_list(torch, elems=512):
    """An AdamW object whose read calls go nowhere."""
    import contextlib
    import types
    cuda = types.SimpleNamespace(stream=lambda s: contextlib.nullcontext(), current_stream=lambda device=None: None)
    opt = bd.AdamW.__new__(bd.AdamW)
    opt.device, opt._index, opt.moment_elems, opt._ctx = torch.device("cuda", 0), 0, elems, None
    opt._cuda, opt._device, opt._current, opt._streams = cuda, lambda: 0, lambda index: 7, {7}
    opt._ws_at, opt._ws_bytes, opt._held = 0, 0, []
    opt._dtypes = {torch.float32: bd.DTYPE_F32, torch.bfloat16: bd.DTYPE_BF16}
    opt.calls = []

    def call(*args):
        opt.calls.append(args)
        return 0

    opt._read = opt._step = call
    return opt, cuda


@pytest.mark.parametrize("given", ["m", "v", "mv", ""])
@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_the_moment_that_is_not_given_takes_the_type_of_the_other(monkeypatch, given, kind):
    torch = pytest.importorskip("torch")
    opt, cuda = fake_list(torch)
    monkeypatch.setattr(torch, "cuda", cuda)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: FakeMemory(n, dtype, None))
    kind = getattr(torch, kind)
    for dtype in (None, kind):
        passed = {k: FakeMemory(512, kind, None) for k in given}
        out = opt.read_moments(dtype, **passed)
        want = kind if given or dtype is not None else torch.float32
        assert [t.dtype for t in out] == [want, want] and opt.calls[-1][3] == opt._dtypes[want]
    if given:
        other = torch.float32 if kind is torch.bfloat16 else torch.bfloat16
        with pytest.raises(ValueError):
            opt.read_moments(other, **{k: FakeMemory(512, kind, None) for k in given})


@pytest.mark.parametrize("step", [1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 32), -(1 << 32) + 3])
def test_step_numbers_are_not_cut_to_32_bits(step):
    # 2^32 would continue the counter, 2^32 + 5 be step 5
    torch = pytest.importorskip("torch")
    opt, _ = fake_list(torch)
    opt.step(1e-3, step=(1 << 31) - 1)
    assert opt.calls[-1][1] == (1 << 31) - 1
    with pytest.raises(ValueError, match="32-bit"):
        opt.step(1e-3, step=step)
    assert len(opt.calls) == 1

    class Param(FakeMemory):
        device, shape, is_contiguous = torch.device("cuda", 0), (512,), lambda self: True

    p, g = Param(512, torch.float32, None), Param(512, torch.float32, None)
    with pytest.raises(ValueError, match="steps_taken"):
        bd.AdamW([p], [g], steps_taken=step)


def test_a_refused_tensor_is_named_by_its_place_in_the_list():
    torch = pytest.importorskip("torch")

    class Tensor(FakeMemory):
        device = torch.device("cuda", 0)

        def __init__(self, shape=(512,), dtype=torch.float32):
            super().__init__(512, dtype, None)
            self.shape = shape

    lists = dict(params=[Tensor() for _ in range(3)], grads=[Tensor() for _ in range(3)], m=[Tensor() for _ in range(3)])
    with pytest.raises(ValueError, match=r"copies\[2\] must be"):
        bd.AdamW(**lists, v=lists["m"], copies=[None, None, Tensor()])
    with pytest.raises(ValueError, match=r"copies\[2\] has shape"):
        bd.AdamW(**lists, v=lists["m"], copies=[Tensor(dtype=torch.bfloat16), None, Tensor((2, 256), torch.float16)])
    eight = [Tensor(), Tensor(dtype=torch.uint8), Tensor(dtype=torch.uint8)]
    bad = Tensor((2,), torch.uint8)
    bad.n, bad.is_contiguous = 2, lambda: False
    with pytest.raises(ValueError, match=r"m_scale\[2\] must be"):
        good = Tensor((2,), torch.uint8)
        good.n = 2
        bd.AdamW(lists["params"], lists["grads"], m=eight, v=eight, m_scale=[None, good, bad], state_bits=[32, 8, 8])


def test_the_longest_tensors(lib):
    # addresses are not touched; a gradient list describes 2^38 elements in chunks, 256 MB on the host
    rc, ctx, _ = grads_init(lib, [(1 << 38, 1 << 40, bd.DTYPE_BF16)])
    assert rc == bd.SHAMPOO_OK
    lib.shampoo_grads_destroy(ctx)
    assert grads_init(lib, [((1 << 38) + 1, 1 << 40, bd.DTYPE_BF16)])[0] == bd.SHAMPOO_EINVAL
    at = dict(param=1 << 40, grad=2 << 40, m=3 << 40, v=4 << 40)
    for extra in ({}, dict(state_bits=8, m_scale=5 << 40, v_scale=6 << 40)):
        rc, ctx, _, elems = adamw_init(lib, [tensor(n=1 << 38, **at, **extra)])
        assert rc == bd.SHAMPOO_OK and elems == 1 << 38
        lib.shampoo_adamw_destroy(ctx)
        more = {k: v + (1 << 43) for k, v in {**at, **extra}.items() if k != "state_bits"}
        if extra:
            more["state_bits"] = 8
        for rows in ([tensor(n=(1 << 38) + 1, **at, **extra)],
                     [tensor(n=1 << 38, **at, **extra), tensor(n=1 << 38, **more)]):
            assert adamw_init(lib, rows)[0] == bd.SHAMPOO_EINVAL  # too long, or the list is


@pytest.mark.parametrize("root", ["newton_db", "chebyshev", "coupled_newton", "newton_db_static"])
def test_roots_come_from_the_memory_of_the_stream_that_writes_them(monkeypatch, root):
    torch = pytest.importorskip("torch")
    import contextlib
    import types
    ours, side = (types.SimpleNamespace(cuda_stream=h) for h in (7, 8))
    current = [ours]

    @contextlib.contextmanager
    def stream(s):
        current.append(current[-1] if s is None else s)
        yield
        current.pop()

    calls = []

    def call(*args):
        calls.append(args)
        return 0

    fake = types.SimpleNamespace(stream=stream, current_stream=lambda device=None: current[-1])
    fresh = lambda *a, **kw: FakeMemory(1024, None, current[-1])
    lib = types.SimpleNamespace(shampoo_inv_root_workspace_bytes=lambda *a: 1024, **{f"shampoo_inv_root_{root}": call})
    monkeypatch.setattr(bd, "_lib", lib)
    monkeypatch.setattr(torch, "cuda", fake)
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, fresh)
    A = FakeMemory(1024, torch.float32, ours)
    A.shape, A.device = (1, 32, 32), None
    for s in (None, side):
        for given in ({}, {"X": FakeMemory(1024, None, ours)}):
            out = getattr(bd, f"inv_root_{root}")(A, FakeMemory(1, None, ours), stream=s, **given)
            assert calls[-1][-1].value == (7 if s is None else 8) and current == [ours]
            for t in out:
                if t is given.get("X"):
                    assert not t.recorded
                else:
                    assert t.on is (ours if s is None else side) and t.recorded == ([] if s is None else [ours])
