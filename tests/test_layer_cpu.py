"""The entry points that run a calibrated layer, without a GPU: validation in the library, buffer
checks in the binding, the calls that calibrate makes for packed weights, and the reference itself."""
import ctypes
import types

import pytest
import torch

import scale_calibration_lh_b200 as L
from tests import layer_ref as R
from tests.test_binding_cpu import _Recorder, fake_streams  # noqa: F401  (fixture)

PTR = ctypes.c_void_p(256)
E4M3 = torch.float8_e4m3fn


@pytest.fixture
def fake(monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(L, "_lib", rec)
    monkeypatch.setattr(L, "_raw_stream", lambda stream: 0)
    return rec


@pytest.fixture(scope="module")
def lib():
    from scale_calibration_lh_b200 import build

    build.build()
    return L.load_library()


def _err(lib):
    return lib.lhcal_last_error_string().decode()


def test_pack_and_unpack_validate(lib):
    f = lib.lhcal_pack_weights
    assert f(2, PTR, 1, 4, 32, PTR, PTR, PTR, None) == L.ERR_UNSUPPORTED  # E4M3 weights
    assert f(1, PTR, 1, 4, 40, PTR, PTR, PTR, None) == L.ERR_INVALID_ARG and "multiple of 16" in _err(lib)
    assert f(1, PTR, 0, 4, 32, PTR, PTR, PTR, None) == L.ERR_INVALID_ARG
    assert f(1, PTR, 1, 0, 32, PTR, PTR, PTR, None) == L.ERR_INVALID_ARG
    assert f(1, PTR, 1, 2 ** 31, 32, PTR, PTR, PTR, None) == L.ERR_INVALID_ARG
    assert f(1, None, 1, 4, 32, PTR, PTR, PTR, None) == L.ERR_INVALID_ARG and "w is NULL" in _err(lib)
    u = lib.lhcal_unpack_weights
    assert u(PTR, PTR, PTR, 1, 4, 32, None, None, None) == L.ERR_INVALID_ARG and "wq16" in _err(lib)
    assert u(PTR, PTR, PTR, 1, 4, 0, PTR, None, None) == L.ERR_INVALID_ARG
    assert u(ctypes.c_void_p(260), PTR, PTR, 1, 4, 32, PTR, None, None) == L.ERR_INVALID_ARG
    assert "aligned" in _err(lib)


def _matvec(lib, **kw):
    a = dict(xtype=L.BF16, x=PTR, x_scale=None, scale_block=0, x_rows=2, ldx=64, experts=None, slots=2, groups=1, rows=8,
             cin=64, packed=PTR, codes=PTR, g=PTR, ytype=L.F32, y=PTR, ldy=8, stream=None)
    a.update(kw)
    return lib.lhcal_matvec(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(xtype=L.F32), L.ERR_UNSUPPORTED, "E4M3"),
    (dict(ytype=L.E4M3), L.ERR_UNSUPPORTED, "y"),
    (dict(cin=40, ldx=64), L.ERR_INVALID_ARG, "multiple of 16"),
    (dict(cin=65536 * 16, ldx=65536 * 16), L.ERR_INVALID_ARG, "too large"),
    (dict(rows=0), L.ERR_INVALID_ARG, "rows"),
    (dict(groups=2), L.ERR_INVALID_ARG, "experts"),
    (dict(slots=4), L.ERR_INVALID_ARG, "x_rows"),
    (dict(x_rows=65, slots=65), L.ERR_INVALID_ARG, "at most 64"),
    (dict(x_rows=-1, slots=-1), L.ERR_INVALID_ARG, "negative"),
    (dict(scale_block=128), L.ERR_INVALID_ARG, "only for E4M3"),
    (dict(x_scale=PTR), L.ERR_INVALID_ARG, "only for E4M3"),
    (dict(xtype=L.E4M3, scale_block=64, x_scale=PTR), L.ERR_INVALID_ARG, "scale_block"),
    (dict(ldx=48), L.ERR_INVALID_ARG, "strides"),
    (dict(ldx=68), L.ERR_INVALID_ARG, "16 bytes"),
    (dict(xtype=L.E4M3, x_scale=PTR, ldx=72), L.ERR_INVALID_ARG, "16 bytes"),
    (dict(ldy=7), L.ERR_INVALID_ARG, "strides"),
    (dict(experts=PTR, slots=1025, x_rows=1025), L.ERR_INVALID_ARG, "at most 1024"),
    (dict(experts=PTR, slots=5), L.ERR_INVALID_ARG, "multiple of x_rows"),
    (dict(experts=PTR, slots=5, x_rows=0), L.ERR_INVALID_ARG, "multiple of x_rows"),
    (dict(x=None), L.ERR_INVALID_ARG, "x is NULL"),
    (dict(x=ctypes.c_void_p(264)), L.ERR_INVALID_ARG, "aligned"),
])
def test_matvec_validates(lib, kw, status, word):
    assert _matvec(lib, **kw) == status and word in _err(lib)


Y0 = 1 << 20  # of the calls below: fp32 y [2, 8], 64 bytes in all


@pytest.mark.parametrize("kw,word", [
    (dict(x=Y0), "y overlaps x"), (dict(x=Y0 - 240), "y overlaps x"), (dict(x=Y0 - 256), None), (dict(x=Y0 + 64), None),
    (dict(packed=Y0 + 56), "y overlaps packed"), (dict(packed=Y0 - 248), "y overlaps packed"), (dict(packed=Y0 - 256), None),
    (dict(codes=Y0 - 31), "y overlaps codes"), (dict(codes=Y0 - 32), None), (dict(g=Y0 + 60), "y overlaps g"),
    (dict(g=Y0 - 4), None), (dict(experts=Y0 - 8), None), (dict(experts=Y0 - 4), "y overlaps experts"),
    (dict(xtype=L.E4M3, x_scale=Y0 - 4), "y overlaps x_scale"), (dict(xtype=L.E4M3, x_scale=Y0 - 8), None),
    (dict(experts=1 << 28, groups=65535, rows=2 ** 31 - 1, cin=65535 * 16, ldx=65535 * 16, ldy=2 ** 31, packed=Y0 + (1 << 36)), "overlaps"),
    (dict(x=Y0 + 32, ldx=80, ldy=40), None),  # x and y as columns of one buffer
    (dict(x=Y0 + 16, ldx=80, ldy=40), "y overlaps x"),
])
def test_matvec_refuses_overlaps(lib, kw, word):
    """A CTA reads its inputs while another writes y. None: no overlap, so that the call goes on to the
    pointers, which are no device memory here."""
    at = dict(x=1 << 24, packed=1 << 25, codes=1 << 26, g=1 << 27, y=Y0)
    at.update(kw)
    assert _matvec(lib, **{k: ctypes.c_void_p(v) if k in ("x", "x_scale", "packed", "codes", "g", "experts", "y") else v
                           for k, v in at.items()}) == L.ERR_INVALID_ARG
    assert (word or "device memory") in _err(lib) or (word is None and "query pointer" in _err(lib)), _err(lib)


def test_matvec_without_tokens_checks_sizes_only(lib):
    none = dict(x_rows=0, slots=0, x=None, y=None, packed=None, codes=None, g=None)
    assert _matvec(lib, **none) == L.OK
    assert _matvec(lib, experts=PTR, **none) == L.OK
    assert _matvec(lib, **{**none, "cin": 8}) == L.ERR_INVALID_ARG


@pytest.mark.parametrize("groups", [1, 3, 512])
@pytest.mark.parametrize("n", [0, 2])
def test_routed_call_without_slots_through_the_binding(lib, monkeypatch, groups, n):
    """A step whose batch is empty: an empty tensor of experts has no address, and is not a missing one."""
    monkeypatch.setattr(L, "_raw_stream", lambda stream: 0)
    packed, codes = torch.zeros(groups, 8, 32, dtype=torch.uint8), torch.zeros(groups, 8, 4, dtype=torch.uint8)
    x, y = torch.zeros(n, 64, dtype=torch.bfloat16), torch.zeros(0, 8)
    e = torch.zeros(0, dtype=torch.int32)
    L.lhcal_matvec(x, packed, codes, torch.ones(groups), y, experts=e)
    q = torch.zeros(n, 64, dtype=E4M3)
    L.lhcal_matvec(q, packed, codes, torch.ones(groups), y, experts=e.view(0, 1), x_scale=torch.ones(n, 1))
    with pytest.raises(ValueError):
        L.lhcal_matvec(x, packed, codes, torch.ones(groups), torch.zeros(1, 8), experts=e)
    if n == 0 and groups == 1:
        L.lhcal_matvec(x, packed, codes, torch.ones(1), y)


def _norm(lib, **kw):
    a = dict(dtype=L.BF16, x=ctypes.c_void_p(1 << 20), tokens=4, cin=64, ldx=64, residual=None, ldr=64, residual_out=None,
             ldro=64, wtype=L.BF16, weight=None, eps=1e-6, y=ctypes.c_void_p(1 << 21), ldy=64, y8=None, ldy8=64,
             y8_scale=None, scale_block=0, stream=None)
    a.update(kw)
    return lib.lhcal_rmsnorm(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(dtype=L.E4M3), L.ERR_UNSUPPORTED, "dtype"),
    (dict(wtype=5), L.ERR_UNSUPPORTED, "dtype"),
    (dict(cin=24, ldx=24), L.ERR_INVALID_ARG, "multiple of 16"),
    (dict(tokens=-1), L.ERR_INVALID_ARG, "tokens"),
    (dict(tokens=2 ** 31), L.ERR_INVALID_ARG, "tokens"),
    (dict(eps=-1.0), L.ERR_INVALID_ARG, "eps"),
    (dict(eps=float("nan")), L.ERR_INVALID_ARG, "eps"),
    (dict(eps=float("inf")), L.ERR_INVALID_ARG, "eps"),
    (dict(residual_out=PTR), L.ERR_INVALID_ARG, "residual"),
    (dict(y=None), L.ERR_INVALID_ARG, "both NULL"),
    (dict(y8=PTR), L.ERR_INVALID_ARG, "y8_scale"),
    (dict(y8_scale=PTR), L.ERR_INVALID_ARG, "y8_scale"),
    (dict(scale_block=128), L.ERR_INVALID_ARG, "only for y8"),
    (dict(scale_block=16), L.ERR_INVALID_ARG, "scale_block"),
    (dict(ldx=48), L.ERR_INVALID_ARG, "stride"),
    (dict(ldx=68), L.ERR_INVALID_ARG, "stride"),
    (dict(ldy=60), L.ERR_INVALID_ARG, "stride"),
    (dict(x=None), L.ERR_INVALID_ARG, "x is NULL"),
])
def test_rmsnorm_validates(lib, kw, status, word):
    assert _norm(lib, **kw) == status and word in _err(lib)


X, Y = 1 << 20, 1 << 21  # of _norm: 4 rows of 64 channels


@pytest.mark.parametrize("kw,word", [
    (dict(weight=Y), "y overlaps weight"), (dict(weight=Y + 256), "y overlaps weight"),
    (dict(weight=Y - 112), "y overlaps weight"),
    (dict(weight=Y - 240, wtype=L.F32), "y overlaps weight"),
    (dict(y8=1 << 22, y8_scale=(1 << 22) + 16), "y8 overlaps y8_scale"),
    (dict(y8=1 << 22, y8_scale=Y + 508), "y overlaps y8_scale"),
    (dict(y8=1 << 22, y8_scale=X), "y8_scale overlaps x"),
    (dict(y8=1 << 22, y8_scale=Y - 16, scale_block=128, ldy=128, cin=128, ldx=128, ldy8=128), None),
    (dict(y8=1 << 22, weight=1 << 23, y8_scale=(1 << 23) + 124), "y8_scale overlaps weight"),
    (dict(y8=1 << 22, weight=1 << 23, y8_scale=(1 << 23) + 128), None),
    (dict(residual=1 << 24, residual_out=1 << 25, weight=1 << 25), "residual_out overlaps weight"),
    (dict(weight=X), None), (dict(weight=Y - 128), None), (dict(weight=Y + 512), None),  # inputs may share; next to y
    (dict(weight=Y + 128, ldy=128), None),  # between two rows of y
    (dict(weight=Y + 256 * 3 + 112, ldy=128), "y overlaps weight"), (dict(weight=Y + 256 * 3 + 128, ldy=128), None),
    (dict(y8=Y + 128, y8_scale=1 << 22, ldy=128, ldy8=256), None),  # rows of y8 in every gap of y
    (dict(y8=Y + 128, y8_scale=1 << 22, ldy=128, ldy8=512), None),  # in every second one
    (dict(y8=Y + 128, y8_scale=1 << 22, ldy=128, ldy8=144), "overlaps"),
    (dict(ldx=0), "stride"), (dict(ldy=-64), "stride"),
    (dict(residual=Y + 128, residual_out=Y + 128, ldr=128, ldro=128, ldy=128), None),  # columns of one buffer
    (dict(residual=Y + 112, residual_out=Y + 112, ldr=128, ldro=128, ldy=128), "overlaps"),
])
def test_rmsnorm_refuses_overlaps_of_all_its_tensors(lib, monkeypatch, kw, word):
    """Outputs against the weight and the scales, too. None: no overlap, so that the call goes on to the
    pointers, which are no device memory here."""
    kw = {k: ctypes.c_void_p(v) if k in ("weight", "y8", "y8_scale", "residual", "residual_out") else v for k, v in kw.items()}
    assert _norm(lib, **kw) == L.ERR_INVALID_ARG
    assert (word or "device memory") in _err(lib) or (word is None and "query pointer" in _err(lib)), _err(lib)


def test_rmsnorm_without_tokens(lib):
    assert _norm(lib, tokens=0, x=None) == L.OK


@pytest.mark.parametrize("block", [0, 128])
def test_rmsnorm_without_tokens_through_the_binding(lib, monkeypatch, block):
    """Outputs of no rows have no address, and are not missing ones."""
    monkeypatch.setattr(L, "_raw_stream", lambda stream: 0)
    x = torch.zeros(0, 192, dtype=torch.bfloat16)
    y8, s = torch.zeros(0, 192, dtype=E4M3), torch.zeros(0, R.scale_blocks(192, block))
    L.lhcal_rmsnorm(x, y=torch.zeros_like(x))
    L.lhcal_rmsnorm(x, torch.ones(192), residual=x, residual_out=torch.zeros_like(x), y=torch.zeros_like(x), y8=y8, y8_scale=s,
                    scale_block=block)
    L.lhcal_rmsnorm(x, y8=y8, y8_scale=s, scale_block=block)
    for bad in (dict(), dict(y8=y8), dict(y=x, y8_scale=s), dict(y=x, residual_out=x)):
        with pytest.raises(L.LhcalError):
            L.lhcal_rmsnorm(x, **bad)


def test_binding_rejects_what_the_library_would_misread(fake):
    packed, codes, g = torch.zeros(2, 8, 32, dtype=torch.uint8), torch.zeros(2, 8, 4, dtype=torch.uint8), torch.ones(2)
    x, y = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(6, 8)
    e = torch.zeros(6, dtype=torch.int32)
    L.lhcal_matvec(x, packed, codes, g, y, experts=e)
    (args,) = fake.args("lhcal_matvec")
    assert args[0] == L.BF16 and args[3:6] == (0, 3, 64) and args[7:11] == (6, 2, 8, 64) and args[16] == 8
    good = dict(x=x, packed=packed, codes=codes, g=g, y=y, experts=e)
    for bad, exc in [(dict(x=x.float()), TypeError), (dict(x=x[:, :48]), ValueError), (dict(x=x.t()), ValueError),
                     (dict(codes=codes[:, :, :3]), ValueError), (dict(codes=codes.int()), TypeError),
                     (dict(g=g[:1]), ValueError), (dict(y=y[:5]), ValueError), (dict(y=y.double()), TypeError),
                     (dict(y=torch.zeros(8, 6).t()), ValueError), (dict(experts=e.long()), TypeError),
                     (dict(experts=torch.zeros(12, dtype=torch.int32)[::2]), ValueError),
                     (dict(packed=packed[0]), ValueError), (dict(packed=packed[:, ::2]), ValueError)]:
        with pytest.raises(exc):
            L.lhcal_matvec(**{**good, **bad})
    q = torch.zeros(3, 192, dtype=E4M3)
    p3, c3 = torch.zeros(1, 8, 96, dtype=torch.uint8), torch.zeros(1, 8, 12, dtype=torch.uint8)
    with pytest.raises(ValueError):  # two scales a row are needed
        L.lhcal_matvec(q, p3, c3, g, torch.zeros(3, 8), x_scale=torch.ones(3, 1), scale_block=128)
    n = torch.zeros(3, 192, dtype=torch.bfloat16)
    for bad, exc in [(dict(residual=n.float()), TypeError), (dict(residual=n[:2]), ValueError), (dict(y=n[:, :96]), ValueError),
                     (dict(y8=n), TypeError), (dict(weight=torch.ones(100)), ValueError),
                     (dict(y8=q, y8_scale=torch.ones(3, 1), scale_block=128), ValueError),
                     (dict(weight=torch.ones(192, dtype=torch.float16)), TypeError)]:
        with pytest.raises(exc):
            L.lhcal_rmsnorm(n, **{"y": torch.zeros_like(n), **bad})
    w = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        L.lhcal_pack_weights(w, g, codes, packed[:1])
    with pytest.raises(ValueError):
        L.lhcal_unpack_weights(packed, codes, g, wq=torch.zeros(1, 8, 64))


def test_scales_of_another_block_are_rejected(fake):
    """[n, C / 128] scales with the default of one a row (or the reverse) would be read as other rows' scales."""
    packed, codes, g = torch.zeros(1, 8, 128, dtype=torch.uint8), torch.zeros(1, 8, 16, dtype=torch.uint8), torch.ones(1)
    q, n = torch.zeros(3, 256, dtype=E4M3), torch.zeros(3, 256, dtype=torch.bfloat16)
    for cols, block in ((2, 0), (3, 128), (1, 128)):
        s = torch.ones(3, cols)
        with pytest.raises(ValueError):
            L.lhcal_matvec(q, packed, codes, g, torch.zeros(3, 8), x_scale=s, scale_block=block)
        with pytest.raises(ValueError):
            L.lhcal_rmsnorm(n, y8=q, y8_scale=s, scale_block=block)
    assert not fake.names()
    for s, block in ((torch.ones(3, 1), 0), (torch.ones(3), 0), (torch.ones(64, 1), 0), (torch.ones(3, 2), 128),
                     (torch.ones(64, 2), 128), (torch.ones(6), 128), (torch.ones(1, 3), 0)):
        L.lhcal_matvec(q, packed, codes, g, torch.zeros(3, 8), x_scale=s, scale_block=block)
        L.lhcal_rmsnorm(n, y8=q, y8_scale=s, scale_block=block)


def test_one_row_passes_no_stride(fake):
    """A single row of a wider (or oddly strided) buffer is dense whatever its stride says."""
    packed, codes, g = torch.zeros(1, 8, 32, dtype=torch.uint8), torch.zeros(1, 8, 4, dtype=torch.uint8), torch.ones(1)
    x = torch.zeros(64, dtype=torch.bfloat16).as_strided((1, 64), (1, 1))
    L.lhcal_matvec(x, packed, codes, g, torch.zeros(1, 8))
    assert fake.args("lhcal_matvec")[0][5] == 64


def test_calibrate_packs_when_the_buffers_ask(fake):
    w = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    b = L.Buffers("mse", 0, 64, 8, 2, L.BF16, "cpu", want_packed=True)
    L.calibrate("mse", None, w, buffers=b)
    assert fake.names() == ["lhcal_global_scale", "lhcal_scale_sweep", "lhcal_pack_weights"]
    (a,) = fake.args("lhcal_pack_weights")
    assert a[0] == L.BF16 and a[2:5] == (2, 8, 64)
    assert [p.value for p in (a[1], a[5], a[6], a[7])] == [t.data_ptr() for t in (w, b.g, b.codes, b.packed)]


@pytest.mark.parametrize("groups,rows", [(3, 8), (1, 300)])
def test_calibrate_host_packs_each_chunk(fake, fake_streams, groups, rows):
    w = torch.zeros(groups, rows, 32, dtype=torch.bfloat16)
    b = L.Buffers("mse", 0, 32, rows, groups, L.BF16, "cpu", want_packed=True)
    b.packed.fill_(3)
    out = types.SimpleNamespace(codes=torch.zeros_like(b.codes), g=torch.zeros_like(b.g), loss=None, wq=None, wq16=None,
                                packed=torch.zeros_like(b.packed))
    L.calibrate_host("mse", None, w, b, {"w": torch.empty_like(w)}, out=out)
    calls = fake.args("lhcal_pack_weights")
    assert len(calls) == len(fake.args("lhcal_scale_sweep")) == 3
    assert sum(c[2] * c[3] for c in calls) == groups * rows
    assert (out.packed == 3).all()


def test_reference_pack_matches_hand_values():
    """Ties to the even code, the clamp at 6, signs kept on zeros, a zero scale."""
    codes = torch.tensor([[[56, 0]]], dtype=torch.uint8)  # 1.0 and 0
    vals = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 9.0, -0.0, -0.26, 0.74, -1.26, 2.51, 3.49, 5.01, -6.0]
    w = torch.tensor([[vals + [1.0] * 16]])
    want = [0, 2, 2, 4, 4, 6, 6, 7, 8, 9, 1, 11, 5, 5, 7, 15] + [0] * 16
    assert R.pack(w, codes, torch.ones(1))[0, 0].tolist() == want


def test_reference_decodes_the_formats():
    assert R.e4m3_table()[:127].tolist() == torch.arange(127, dtype=torch.uint8).view(E4M3).float().tolist()
    packed = torch.tensor([[0x10, 0xF2] + [0] * 6], dtype=torch.uint8)
    assert R.weight_values(packed, torch.tensor([[57]], dtype=torch.uint8))[0, :4].tolist() == [0.0, 0.5625, 1.125, -6.75]


def test_buffers_scales_begin_defined(monkeypatch, fake):
    """Global scales that no call has written yet compare equal to a copy of them, whatever lay in memory before."""
    empty = torch.empty

    def dirty(*a, **k):
        t = empty(*a, **k)
        return t.fill_(float("nan")) if t.is_floating_point() else t

    monkeypatch.setattr(torch, "empty", dirty)
    b = L.Buffers("mse", 0, 64, 8, 2, L.BF16, "cpu")
    assert torch.equal(b.g, b.g.clone())
