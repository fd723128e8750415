"""Block-scaled operators on the host: the scale order and the references the
GPU tests use, and the calls that are refused before anything is enqueued."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

import oracle
from _block import act_parts, blocks_of, cast_values, codes_of, exponents, packed, round_fp8, scale_address, spread

FAKE = 0x10000  # an address that is never used: every call fails its host checks first


@pytest.fixture(scope="module")
def lib():
    from fp8_mixed_precision_tensor_b200 import build, fp8

    build.build()
    return fp8.load_library()


@pytest.fixture(scope="module")
def fp8():
    from fp8_mixed_precision_tensor_b200 import build, fp8

    build.build()
    return fp8


# ---------------------------------------------------------------- references
@pytest.mark.parametrize("outer,red", [(1, 1), (5, 128), (128, 512), (130, 513), (300, 2000)])
def test_scale_addresses_are_distinct_and_fill_the_buffer(lib, outer, red):
    kb = -(-red // 128)
    r, b = np.meshgrid(np.arange(outer), np.arange(kb), indexing="ij")
    at = scale_address(r, b, red).reshape(-1)
    n = lib.fp8_block_scale_bytes(outer, red)
    assert len(set(at.tolist())) == outer * kb and at.max() < n
    assert n == -(-outer // 128) * -(-kb // 4) * 512
    # whole groups of 128 rows x 4 blocks use every byte
    R, C = -(-outer // 128) * 128, -(-kb // 4) * 512
    r, b = np.meshgrid(np.arange(R), np.arange(C // 128), indexing="ij")
    assert sorted(scale_address(r, b, C).reshape(-1).tolist()) == list(range(n))


def test_scale_bytes_of_empty_operands(lib):
    for outer, red in ((0, 5), (5, 0), (0, 0), (-1, 4), (4, -1)):
        assert lib.fp8_block_scale_bytes(outer, red) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_block_reference_is_the_per_tensor_rule_on_each_block(fmt):
    """The test reference against the oracle's per-tensor scale and cast on every block."""
    code = {"e4m3": oracle.E4M3, "e5m2": oracle.E5M2}[fmt]
    x = np.random.default_rng(3).standard_normal((70, 300)).astype(np.float32)
    x *= np.exp2(np.random.default_rng(4).integers(-40, 40, (70, 300))).astype(np.float32)
    x[3] = 0.0
    v, k = cast_values(x, fmt, 1, 128)
    q = codes_of(v, spread(k, 1, 128, x.shape), fmt)
    for r in range(0, 70, 7):
        for b in range(3):
            blk = np.ascontiguousarray(x[r, b * 128:(b + 1) * 128])
            rc, s = oracle.compute_scale(oracle.amax(blk), code, 0)
            assert rc == 0 and s == 2.0 ** int(k[r, b])
            assert np.array_equal(oracle.cast(blk, code, s), q[r, b * 128:(b + 1) * 128])


def test_rounding_reference_against_torch_and_every_midpoint():
    for fmt, tt, code in (("e4m3", torch.float8_e4m3fn, oracle.E4M3), ("e5m2", torch.float8_e5m2, oracle.E5M2)):
        table = np.array(sorted({abs(float(t)) for t in oracle.decode_table(code) if np.isfinite(t)}))
        mid = (table[1:] + table[:-1]) / 2
        for v in (table, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9)):
            got = round_fp8(v, fmt)
            assert np.all(np.isin(got, table))
            assert np.all(np.abs(got - v) <= np.min(np.abs(table[None] - v[:, None]), axis=1))
        f32 = mid.astype(np.float32)
        assert np.array_equal(round_fp8(f32, fmt), torch.from_numpy(f32).to(tt).double().numpy())


@pytest.mark.parametrize("kind", ["gelu_tanh", "gelu_erf", "silu"])
def test_activation_reference_against_torch_and_differences(kind):
    h = np.linspace(-9, 9, 2001)
    a, d = act_parts(h, kind)
    t = torch.from_numpy(h)
    want = {"gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh"),
            "gelu_erf": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}[kind](t).numpy()
    assert np.max(np.abs(a - want)) < 1e-13
    e = 1e-5
    diff = (act_parts(h + e, kind)[0] - act_parts(h - e, kind)[0]) / (2 * e)
    # a central difference is off by e^2 / 6 of the third derivative (below 3 here) and by the rounding of a / e
    assert np.max(np.abs(d - diff)) < 3 * e * e / 6 + 4 * 9 * 2.0 ** -53 / e


def test_exponents_at_and_beside_the_thresholds():
    a = np.array([[448.0, np.nextafter(448.0, 1e9), 1.75, 0.0, np.inf, 1e-44, 3e38]])
    assert exponents(a, "e4m3").tolist() == [[0, -1, 8, 0, 0, 126, -120]]
    assert packed(np.array([[3]]), 1, 5)[0] == 124 and blocks_of(np.ones((3, 5)), 2, 2).shape == (2, 3)


# ---------------------------------------------------------------- refusals, C ABI
def _b(fp8, q=FAKE, s=FAKE, ld=256):
    return ctypes.byref(fp8._Blocks(q, s, ld))


def test_block_casts_reject_bad_arguments(lib, fp8):
    ok = dict(x=FAKE, dt=1, rows=8, cols=256, ldx=256, fmt=0, margin=0, row=_b(fp8), col=None)

    def call(**kw):
        a = {**ok, **kw}
        return lib.fp8_block_cast(a["x"], a["dt"], a["rows"], a["cols"], a["ldx"], a["fmt"], a["margin"], a["row"],
                                  a["col"], None)

    for kw in (dict(dt=3), dict(dt=9), dict(fmt=2), dict(rows=-1), dict(cols=-1), dict(margin=-1), dict(margin=65),
               dict(row=None), dict(x=None), dict(ldx=255), dict(row=_b(fp8, None)), dict(row=_b(fp8, FAKE, None)),
               dict(row=_b(fp8, ld=240)), dict(col=_b(fp8, None))):
        assert call(**kw) == fp8.FP8_ERR_INVALID_ARG, kw
    for kw in (dict(x=FAKE + 1), dict(row=_b(fp8, FAKE + 8)), dict(row=_b(fp8, FAKE, FAKE + 4)),
               dict(row=_b(fp8, ld=264)), dict(col=_b(fp8, ld=257))):
        assert call(**kw) == fp8.FP8_ERR_UNALIGNED, kw
    assert call(rows=0) == fp8.FP8_OK and call(cols=0) == fp8.FP8_OK  # nothing to do, nothing enqueued
    sq = lib.fp8_block_cast_square
    assert sq(FAKE, 1, 8, 256, 256, 0, 0, _b(fp8), None, None) == fp8.FP8_ERR_INVALID_ARG
    assert sq(FAKE, 1, 8, 256, 256, 0, 0, None, FAKE, None) == fp8.FP8_ERR_INVALID_ARG
    assert sq(FAKE, 1, 8, 256, 256, 0, 0, _b(fp8), FAKE + 2, None) == fp8.FP8_ERR_UNALIGNED
    assert sq(FAKE, 1, 0, 256, 256, 0, 0, None, None, None) == fp8.FP8_OK
    dec = lib.fp8_block_decode
    assert dec(_b(fp8), 0, 2, 8, 256, FAKE, 1, 256, None) == fp8.FP8_ERR_INVALID_ARG   # axis
    assert dec(_b(fp8), 2, 1, 8, 256, FAKE, 1, 256, None) == fp8.FP8_ERR_INVALID_ARG   # format
    assert dec(_b(fp8), 0, 1, 8, 256, FAKE, 1, 200, None) == fp8.FP8_ERR_INVALID_ARG   # row pitch
    assert dec(_b(fp8), 0, 1, 8, 256, FAKE + 1, 1, 256, None) == fp8.FP8_ERR_UNALIGNED


def test_block_products_reject_bad_arguments(lib, fp8):
    b = _b(fp8)
    fwd = lambda x=b, w=b, bias=None, bdt=0, y=FAKE, ydt=1, ld=256, M=64, N=256, K=256: lib.fp8_block_linear_fwd(  # noqa: E731
        x, w, bias, bdt, y, ydt, ld, M, N, K, None)
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(ydt=4), dict(bias=FAKE, bdt=3), dict(y=None), dict(ld=255),
               dict(x=None), dict(w=None), dict(x=_b(fp8, ld=128)), dict(w=_b(fp8, None))):
        assert fwd(**kw) == fp8.FP8_ERR_INVALID_ARG, kw
    for kw in (dict(y=FAKE + 1), dict(x=_b(fp8, FAKE + 8)), dict(w=_b(fp8, ld=260)), dict(bias=FAKE + 1, bdt=1)):
        assert fwd(**kw) == fp8.FP8_ERR_UNALIGNED, kw
    assert fwd(M=0, x=None, y=None) == fp8.FP8_OK and fwd(N=0) == fp8.FP8_OK
    assert lib.fp8_block_linear_dgrad(b, 2, b, FAKE, 1, 256, 64, 256, 256, None) == fp8.FP8_ERR_INVALID_ARG
    assert lib.fp8_block_linear_wgrad(b, 7, b, FAKE, 1, 256, 64, 256, 256, None) == fp8.FP8_ERR_INVALID_ARG
    assert lib.fp8_block_linear_wgrad(_b(fp8, ld=128), 1, b, FAKE, 1, 256, 64, 256, 256, None) == fp8.FP8_ERR_INVALID_ARG
    tok = lambda x=FAKE, dt=1, ldx=256, margin=0, w=b, y=FAKE, ydt=1, ldy=256, M=4, N=256, K=256: lib.fp8_block_linear_tokens(  # noqa: E731
        x, dt, ldx, margin, w, None, 0, y, ydt, ldy, M, N, K, None)
    for kw in (dict(M=fp8.FP8_BLOCK_TOKENS_MAX + 1), dict(M=-1), dict(dt=3), dict(margin=65), dict(x=None),
               dict(ldx=100), dict(w=None), dict(y=None), dict(ldy=4), dict(ydt=9)):
        assert tok(**kw) == fp8.FP8_ERR_INVALID_ARG, kw
    assert tok(x=FAKE + 1) == fp8.FP8_ERR_UNALIGNED and tok(M=0, x=None) == fp8.FP8_OK


def test_activation_calls_reject_bad_arguments(lib, fp8):
    b = _b(fp8)
    fwd = lambda h=FAKE, dt=1, rows=8, cols=256, ld=256, act=0, margin=0, ck=b, a_row=None, a=None, lda=0: lib.fp8_act_fwd(  # noqa: E731
        h, dt, rows, cols, ld, act, margin, ck, a_row, a, lda, None)
    for kw in (dict(act=3), dict(act=-1), dict(dt=3), dict(margin=65), dict(ck=None), dict(h=None), dict(ld=10),
               dict(a=FAKE, lda=10), dict(a_row=_b(fp8, ld=16)), dict(rows=-2)):
        assert fwd(**kw) == fp8.FP8_ERR_INVALID_ARG, kw
    assert fwd(a=FAKE + 1, lda=256) == fp8.FP8_ERR_UNALIGNED and fwd(rows=0, ck=None) == fp8.FP8_OK
    bwd = lambda ck=b, da=FAKE, dt=1, rows=8, cols=256, ld=256, act=0, fmt=1, margin=0, r=b, c=None, a=None, dh=None, lddh=0: (  # noqa: E731
        lib.fp8_act_bwd(ck, da, dt, rows, cols, ld, act, fmt, margin, r, c, a, dh, lddh, None))
    for kw in (dict(r=None), dict(fmt=2), dict(act=5), dict(ck=None), dict(da=None), dict(dh=FAKE, lddh=5),
               dict(c=_b(fp8, None)), dict(a=_b(fp8, ld=64)), dict(cols=-3)):
        assert bwd(**kw) == fp8.FP8_ERR_INVALID_ARG, kw
    assert bwd(c=_b(fp8, FAKE + 4)) == fp8.FP8_ERR_UNALIGNED and bwd(cols=0) == fp8.FP8_OK


@pytest.mark.parametrize("side", [2 ** 31 - 1, 2 ** 31 - 1023])
def test_sides_near_the_end_of_an_int_are_refused(lib, fp8, side):
    """Rounded up to a tile they would pass it."""
    wide = _b(fp8, ld=2 ** 31)
    calls = [lambda r, c: lib.fp8_block_cast(FAKE, 1, r, c, 2 ** 31, 0, 0, wide, None, None),
             lambda r, c: lib.fp8_block_cast(FAKE, 1, r, c, 2 ** 31, 0, 0, None, wide, None),
             lambda r, c: lib.fp8_block_cast_square(FAKE, 1, r, c, 2 ** 31, 0, 0, wide, FAKE, None),
             lambda r, c: lib.fp8_block_decode(wide, 0, 1, r, c, FAKE, 1, 2 ** 31, None),
             lambda r, c: lib.fp8_act_fwd(FAKE, 1, r, c, 2 ** 31, 0, 0, wide, None, None, 0, None),
             lambda r, c: lib.fp8_act_bwd(wide, FAKE, 1, r, c, 2 ** 31, 0, 1, 0, wide, None, None, None, 0, None),
             lambda n, k: lib.fp8_block_linear_tokens(FAKE, 1, 2 ** 31, 0, wide, None, 0, FAKE, 1, 2 ** 31, 4, n, k, None)]
    for call in calls:
        assert call(side, 64) == fp8.FP8_ERR_UNSUPPORTED and call(64, side) == fp8.FP8_ERR_UNSUPPORTED
    for dims in ((side, 64, 64), (64, side, 64), (64, 64, side)):
        assert lib.fp8_block_linear_fwd(wide, wide, None, 0, FAKE, 1, 2 ** 31, *dims, None) == fp8.FP8_ERR_UNSUPPORTED
        for f in (lib.fp8_block_linear_dgrad, lib.fp8_block_linear_wgrad):
            assert f(wide, 1, wide, FAKE, 1, 2 ** 31, *dims, None) == fp8.FP8_ERR_UNSUPPORTED


def test_sides_that_an_int_does_not_hold_are_refused(fp8, monkeypatch):
    """2^32 + 8 rows are not 8 rows."""
    monkeypatch.setattr(fp8, "_device", lambda t, what: -1)
    u8 = dict(dtype=torch.uint8, device="meta")
    x, q, s = torch.empty((2 ** 32 + 8, 1), device="meta"), torch.empty((2 ** 32 + 8, 16), **u8), torch.empty(2 ** 34, **u8)
    y, few = torch.empty((8, 8), device="meta"), torch.empty((8, 1), device="meta")
    w = torch.empty((8, 16), **u8)
    for call in (lambda: fp8.fp8_block_cast(x, 0, 0, q, s), lambda: fp8.fp8_block_cast_square(x, 0, 0, q, s, s),
                 lambda: fp8.fp8_block_decode(q, s, 0, 1, x), lambda: fp8.fp8_act_fwd(x, 0, 0, q, s),
                 lambda: fp8.fp8_act_bwd(q, s, x, 0, dh=x), lambda: fp8.fp8_block_linear_fwd(q, s, w, s, y),
                 lambda: fp8.fp8_block_linear_fwd(w, s, q, s, y), lambda: fp8.fp8_block_linear_tokens(few, q, s, y),
                 lambda: fp8.fp8_block_linear_dgrad(q, s, 1, w, s, y), lambda: fp8.fp8_block_linear_dgrad(w, s, 1, q.t(), s, y),
                 lambda: fp8.fp8_block_linear_wgrad(q, s, 1, w, s, y), lambda: fp8.fp8_block_linear_wgrad(w, s, 1, q.t(), s, y)):
        with pytest.raises(ValueError, match="a side"):
            call()


def test_the_message_of_an_unsupported_shape_names_both_rules(fp8):
    text = fp8.fp8_strerror(fp8.FP8_ERR_UNSUPPORTED)
    assert "multiples of 16" in text and "2^31 - 1024" in text


def test_binding_takes_device_tensors_only(fp8):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensors"):
        fp8.fp8_block_cast(x, fp8.FP8_E4M3, 0, q, s)
    with pytest.raises(ValueError, match="device tensors"):
        fp8.fp8_act_fwd(x, fp8.FP8_ACT_SILU, 0, q, s)
    with pytest.raises(TypeError):
        fp8.fp8_block_cast(x.double(), fp8.FP8_E4M3, 0, q, s)


def test_short_route_leaves_host_tensors_and_wrong_arguments(fp8):
    x, q, s = torch.zeros(4, 128), torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    assert fp8._calls.block_cast(x, 0, 0, q, s, None, None, None) is False
    assert fp8._calls.block_cast(x, 0, 0) is False and fp8._calls.linear_fwd(*range(8)) is False
    assert fp8._calls.act_fwd(None, 0, 0, q, s, None, None, None, None) is False
    with pytest.raises(TypeError):
        fp8._calls.bind(1, 2)
    with pytest.raises(ValueError):
        fp8._calls.bind(*[0] * 8)


@pytest.mark.parametrize("how", ["missing", "no library", "another torch"])
def test_the_library_serves_without_the_short_route(lib, fp8, monkeypatch, tmp_path, how):
    path = tmp_path / "_calls.so"
    if how == "no library":
        path.write_bytes(b"not a library")
    if how == "another torch":
        monkeypatch.setattr(torch, "__version__", "1.0")
    else:
        monkeypatch.setattr(fp8, "CALLS_PATH", str(path))
    monkeypatch.setattr(fp8, "_lib", None)
    monkeypatch.setattr(fp8, "_calls", None)
    with pytest.warns(RuntimeWarning, match="longer way through Python"):
        assert fp8.fp8_strerror(0) == "ok"
    assert fp8.fp8_adam_workspace_bytes(3) == 3 * 64
    x, q, s = torch.zeros(4, 128), torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    assert fp8._calls.block_cast(x, 0, 0, q, s, None, None, None) is False
    with pytest.raises(ValueError, match="device tensors"):  # the Python function's own answer
        fp8.fp8_block_cast(x, 0, 0, q, s)


# ---------------------------------------------------------------- modules: memory in use on a given stream
class _Stream:
    """In place of torch.cuda.Stream."""


class _Tensor:
    """A tensor of which only the streams that it is recorded on matter."""

    def __init__(self, *shape):
        self.shape, self.used, self.device, self.dtype = shape, set(), "cuda:0", torch.bfloat16

    def record_stream(self, stream):
        self.used.add(stream)


@pytest.fixture
def side(fp8, monkeypatch):
    """A second stream, with the library's calls and torch's allocations left out."""
    now = [_Stream()]

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: now[-1])
    monkeypatch.setattr(torch, "empty", lambda shape, **k: _Tensor(*shape))
    monkeypatch.setattr(fp8, "_stream", lambda s: id(now[-1]))
    monkeypatch.setattr(fp8, "block_codes", lambda rows, cols, device: _Tensor(rows, cols))
    monkeypatch.setattr(fp8, "block_scales", lambda outer, red, device: _Tensor(outer * red))
    for name in ("fp8_block_cast_square", "fp8_block_cast", "fp8_block_linear_tokens", "fp8_block_linear_fwd",
                 "fp8_block_linear_dgrad", "fp8_block_linear_wgrad", "fp8_act_fwd", "fp8_act_bwd"):
        monkeypatch.setattr(fp8, name, lambda *a, **k: None)
    return _Stream()


def test_a_weight_update_holds_its_memory_for_its_stream(side):
    from fp8_mixed_precision_tensor_b200.block_linear import BlockWeight

    w, new = BlockWeight(_Tensor(256, 128)), _Tensor(256, 128)
    w.update(new, stream=side)
    for t in (new, w.q, w.s, w.s_col):
        assert t.used == {side}


@pytest.mark.parametrize("given", [True, False])
def test_passes_hold_the_layers_memory_for_their_stream(side, given):
    from fp8_mixed_precision_tensor_b200.block_linear import BlockLinear, BlockMLP

    def there(f, *a, **k):
        if given:
            return f(*a, **k, stream=side)
        with torch.cuda.stream(side):
            return f(*a, **k)

    for M, keep in ((4, False), (200, False), (200, True)):
        lin = BlockLinear(_Tensor(256, 128), _Tensor(256))
        x = _Tensor(M, 128)
        there(lin.forward, x, keep=keep)
        for t in (lin.weight.q, lin.weight.s, lin.bias, *((x,) if given else ())):
            assert t.used == {side}
    lin = BlockLinear(_Tensor(256, 128))  # no bias; forward here, backward there
    lin.forward(_Tensor(200, 128), keep=True)
    kept = lin.kept.tensors
    assert not any(t.used for t in (*kept, lin.weight.q, lin.weight.s, lin.weight.s_col))
    there(lin.backward, _Tensor(200, 256))
    assert all(t.used == {side} for t in (*kept, lin.weight.q, lin.weight.s_col))
    for there_first in (True, False):
        mlp = BlockMLP(_Tensor(256, 128), _Tensor(64, 256))
        (there if there_first else lambda f, x: f(x))(mlp.forward, _Tensor(200, 128))
        kept = mlp.kept.tensors
        there(mlp.backward, _Tensor(200, 64))
        for w in (mlp.w1, mlp.w2):
            assert all(t.used == {side} for t in (w.q, w.s, w.s_col))
        assert all(t.used == (set() if there_first else {side}) for t in kept)
