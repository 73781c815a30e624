"""Host-side tests of the paged 8-bit cache: argument checks before any CUDA
call, workspace sizes, and the plain implementations the GPU tests use against
closed forms."""
import math
import os
import shutil
import subprocess
import sys

import pytest
import torch

from tests import _paged_ref as ref


@pytest.fixture(scope="module")
def fl():
    from io_aware_exact_34_b200 import build
    build.build()
    from io_aware_exact_34_b200 import fattn
    return fattn


def test_native_calls_are_loaded(fl):
    """Where they can be built they are, and they are the ones in use."""
    from io_aware_exact_34_b200 import build, calls_path
    assert build.build_calls() == calls_path(torch.__version__) == fl._calls.__file__
    assert torch.__version__ in os.path.basename(fl._calls.__file__)


def test_native_calls_that_do_not_load(fl, tmp_path):
    """No file, or one that is no module: the binding goes without."""
    assert fl._load_calls(str(tmp_path / "none.so")) is None
    broken = tmp_path / "broken.so"
    broken.write_bytes(b"no shared object")
    with pytest.warns(UserWarning, match="broken.so does not load"):
        assert fl._load_calls(str(broken)) is None


def test_binding_imports_without_native_calls(fl, tmp_path):
    """The package with its library alone (another torch's native calls beside it are not touched)."""
    from io_aware_exact_34_b200 import build
    pkg = tmp_path / "io_aware_exact_34_b200"
    pkg.mkdir()
    for f in os.listdir(build.PKG):
        if f.endswith(".py"):
            shutil.copy(os.path.join(build.PKG, f), pkg)
    os.symlink(build.LIB, pkg / "libfattn.so")
    for f in ("_fattn_calls.so", "_fattn_calls.torch-0.0.so"):
        (pkg / f).write_bytes(b"no shared object")
    code = "from io_aware_exact_34_b200 import fattn; print(fattn._calls, fattn.attn_decode_paged_fp8_auto_splits(1, 8, 8, 64, 128))"
    res = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout.split() == ["None", "1"], res.stderr


def test_library_builds_without_torch(fl, monkeypatch):
    from io_aware_exact_34_b200 import build
    built = []
    monkeypatch.setattr(build, "build_lib", lambda force, verbose: built.append(force) or build.LIB)
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    with pytest.raises(RuntimeError, match="torch does not import"):
        build.build_calls(force=True)
    with pytest.warns(UserWarning, match="torch does not import"):
        assert build.build(force=True) == build.LIB and built == [True]


A = [0x100000 * (i + 1) for i in range(12)]  # never dereferenced: every call below fails validation first


def _plan(fl, **kw):
    a = dict(lens=A[0], new=A[1], B=4, free=A[2], nfree=8, table=A[3], width=4, page=16, slots=A[4], room=64, cu=A[5],
             out=A[6], counts=A[7])
    a.update(kw)
    return fl.lib.attn_paged_plan(a["lens"], a["new"], a["B"], a["free"], a["nfree"], a["table"], a["width"], a["page"],
                                  a["slots"], a["room"], a["cu"], a["out"], a["counts"], None)


def test_plan_argument_checks(fl):
    for name in ("lens", "new", "table", "slots", "cu", "out", "counts", "free"):
        assert _plan(fl, **{name: None}) == fl.FATTN_ERR_INVALID_ARG, name
    for bad in (dict(B=0), dict(nfree=-1), dict(width=0), dict(room=0), dict(page=0), dict(page=8), dict(page=24)):
        assert _plan(fl, **bad) == fl.FATTN_ERR_INVALID_ARG, bad
    assert _plan(fl, B=16385) == fl.FATTN_ERR_UNSUPPORTED
    for name in ("lens", "new", "free", "table", "cu", "out", "counts"):
        assert _plan(fl, **{name: A[9] + 2}) == fl.FATTN_ERR_MISALIGNED, name
    assert _plan(fl, slots=A[4] + 4) == fl.FATTN_ERR_MISALIGNED
    # outputs over the inputs that are still being read
    for bad in (dict(out=A[0]), dict(out=A[1] + 12), dict(cu=A[0] - 4), dict(cu=A[1])):
        assert _plan(fl, **bad) == fl.FATTN_ERR_INVALID_ARG, bad


def _append(fl, **kw):
    a = dict(k=A[0], v=A[1], ks=256, vs=256, slots=A[2], T=4, kp=A[3], vp=A[4], sk=A[5], sv=A[6], N=4, page=16, H=2, d=128)
    a.update(kw)
    return fl.lib.attn_append_paged_fp8(a["k"], a["v"], a["ks"], a["vs"], a["slots"], a["T"], a["kp"], a["vp"], a["sk"], a["sv"],
                                        a["N"], a["page"], a["H"], a["d"], None)


def test_append_argument_checks(fl):
    for name in ("k", "v", "slots", "kp", "vp", "sk", "sv"):
        assert _append(fl, **{name: None}) == fl.FATTN_ERR_INVALID_ARG, name
    for bad in (dict(T=0), dict(N=0), dict(H=0), dict(page=8), dict(page=17), dict(ks=248), dict(vs=0), dict(ks=-256),
                dict(vp=A[3]), dict(vp=A[3] + 64), dict(sv=A[5] + 28)):
        assert _append(fl, **bad) == fl.FATTN_ERR_INVALID_ARG, bad
    assert _append(fl, d=96) == fl.FATTN_ERR_UNSUPPORTED
    assert _append(fl, H=70000, ks=1 << 30, vs=1 << 30) == fl.FATTN_ERR_UNSUPPORTED
    for bad in (dict(k=A[0] + 8), dict(vp=A[4] + 8), dict(ks=260), dict(sk=A[5] + 2), dict(slots=A[2] + 4)):
        assert _append(fl, **bad) == fl.FATTN_ERR_MISALIGNED, bad


def _attend(fl, fn, **kw):
    a = dict(q=A[0], kp=A[1], vp=A[2], sk=A[3], sv=A[4], table=A[5], width=4, page=16, N=8, o=A[6], lse=A[7], lens=A[8], cu=A[9],
             B=2, T=6, most=4, Hq=4, Hkv=2, d=128, scale=0.1, left=-1, S=4, ws=A[10], bytes=1 << 20)
    a.update(kw)
    head = [a["q"], a["kp"], a["vp"], a["sk"], a["sv"], a["table"], a["width"], a["page"], a["N"], a["o"], a["lse"], a["lens"]]
    if fn == "decode":
        return fl.lib.attn_decode_paged_fp8(*head, a["B"], a["Hq"], a["Hkv"], a["d"], a["scale"], a["left"], a["S"], a["ws"],
                                            a["bytes"], None)
    return fl.lib.attn_fwd_paged_fp8(*head, a["cu"], a["B"], a["T"], a["most"], a["Hq"], a["Hkv"], a["d"], a["scale"], 1, a["left"],
                                     -1, a["ws"], a["bytes"], None)


@pytest.mark.parametrize("fn", ["decode", "fwd"])
def test_attention_argument_checks(fl, fn):
    for name in ("q", "kp", "vp", "sk", "sv", "table", "o", "lens"):
        assert _attend(fl, fn, **{name: None}) == fl.FATTN_ERR_INVALID_ARG, name
    for bad in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(width=0), dict(N=0), dict(page=8), dict(page=48),
                dict(scale=0.0), dict(scale=math.inf), dict(scale=math.nan)):
        assert _attend(fl, fn, **bad) == fl.FATTN_ERR_INVALID_ARG, bad
    for bad in (dict(d=96), dict(Hq=258, Hkv=2), dict(B=65536), dict(width=1 << 28)):
        assert _attend(fl, fn, **bad) == fl.FATTN_ERR_UNSUPPORTED, bad
    for bad in (dict(q=A[0] + 8), dict(kp=A[1] + 8), dict(vp=A[2] + 4), dict(o=A[6] + 2), dict(sk=A[3] + 1), dict(sv=A[4] + 2),
                dict(table=A[5] + 2), dict(lens=A[8] + 2), dict(lse=A[7] + 2)):
        assert _attend(fl, fn, **bad) == fl.FATTN_ERR_MISALIGNED, bad


def test_decode_splits_and_workspace(fl):
    assert _attend(fl, "decode", S=-1) == fl.FATTN_ERR_INVALID_ARG
    assert _attend(fl, "decode", S=65) == fl.FATTN_ERR_INVALID_ARG  # more than the table's 64 keys
    need = fl.attn_decode_workspace_bytes(2, 4, 64, 128, 4)
    assert _attend(fl, "decode", bytes=need - 1) == fl.FATTN_ERR_WORKSPACE
    assert _attend(fl, "decode", ws=None) == fl.FATTN_ERR_WORKSPACE
    assert _attend(fl, "decode", ws=A[10] + 8) == fl.FATTN_ERR_MISALIGNED
    assert fl.attn_decode_paged_fp8_auto_splits(0, 4, 2, 64, 128) == fl.FATTN_ERR_INVALID_ARG
    assert fl.attn_decode_paged_fp8_auto_splits(1, 5, 2, 64, 128) == fl.FATTN_ERR_INVALID_ARG
    for B, Hq, Hkv, Lk in ((1, 32, 8, 16), (1, 32, 8, 1 << 20), (512, 64, 8, 4096), (3, 5, 5, 100)):
        S = fl.attn_decode_paged_fp8_auto_splits(B, Hq, Hkv, Lk, 128)
        assert 1 <= S <= max(1, -(-Lk // 64))


def test_fwd_argument_checks(fl):
    for bad in (dict(cu=None), dict(T=0), dict(most=0)):
        assert _attend(fl, "fwd", **bad) == fl.FATTN_ERR_INVALID_ARG, bad
    assert _attend(fl, "fwd", cu=A[9] + 2) == fl.FATTN_ERR_MISALIGNED
    assert fl.attn_fwd_paged_fp8_workspace_bytes(2, 0, 4, 4, 2, 64, 128) == 0
    assert fl.attn_fwd_paged_fp8_workspace_bytes(2, 6, 4, 4, 3, 64, 128) == 0
    need = fl.attn_fwd_paged_fp8_workspace_bytes(1, 3, 3, 4, 2, 4096, 128)
    assert need > 0 and need % (3 * 4 * 129 * 4) == 0
    assert _attend(fl, "fwd", B=1, T=3, most=3, width=256, bytes=need - 1) == fl.FATTN_ERR_WORKSPACE


def test_integers_beyond_32_bits(fl):
    """Refused where they are sizes; a window of that length is as wide as any."""
    for x in (2 ** 31, 2 ** 32 + 1, -2 ** 31 - 1, 10 ** 30):
        with pytest.raises(ValueError, match="max_tokens"):
            fl._int32(x, "max_tokens")
    assert [fl._int32(x, "") for x in (0, -5, 2 ** 31 - 1, -2 ** 31)] == [0, -5, 2 ** 31 - 1, -2 ** 31]
    for x in (1.0, "3", None):
        with pytest.raises(TypeError):
            fl._int32(x, "max_tokens")
        with pytest.raises(TypeError):
            fl._window(x)
    assert [fl._window(x) for x in (-1, -2 ** 40, 0, 7, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 63 + 5)] == [-1, -1, 0, 7] + [2 ** 31 - 1] * 4
    with pytest.raises(ValueError):
        fl.attn_fwd_paged_fp8_workspace_bytes(1, 2 ** 32 + 8, 8, 8, 8, 64, 128)
    with pytest.raises(ValueError):
        fl.attn_decode_paged_fp8_auto_splits(1, 8, 8, 2 ** 32 + 64, 128)


@pytest.mark.parametrize("d", [64, 128])
def test_more_keys_never_mean_fewer_splits(fl, d):
    """A workspace sized for the whole table serves every window of it."""
    lens = sorted({1 << e for e in range(25)} | {(1 << e) + 1 for e in range(4, 24)} | set(range(100, 40000, 997)))
    for B in (1, 2, 5, 8, 16, 24, 33, 64, 100, 200, 512, 3000):
        for Hq, Hkv in ((8, 8), (32, 8), (16, 1), (71, 1), (10, 2)):
            splits = [fl.attn_decode_paged_fp8_auto_splits(B, Hq, Hkv, n, d) for n in lens]
            assert all(x <= y for x, y in zip(splits, splits[1:])), (B, Hq, Hkv, splits)
            assert all(1 <= x <= 64 and x <= -(-n // 256) for x, n in zip(splits, lens))
            for new in (2, 3, 8):
                if new * (Hq // Hkv) < 49:
                    need = [fl.attn_fwd_paged_fp8_workspace_bytes(B, B * new, new, Hq, Hkv, n, d) for n in lens]
                    assert all(x <= y for x, y in zip(need, need[1:])), (B, Hq, Hkv, new, need)


@pytest.mark.parametrize("d", [64, 128])
def test_long_run_workspace_holds_the_cut_pairs(fl, d):
    """Only the pairs of row tiles of the last, incomplete round of 148 are cut into (at most 32) parts: the workspace of
    a long run has their rows and no others."""
    for B in (1, 2, 3, 5, 16, 64, 300):
        for new in (49, 300, 1984, 2048, 4800, 8192, 30000):
            for Hq, Hkv in ((32, 8), (8, 8), (128, 8), (71, 1), (16, 1), (5, 1), (128, 1)):
                g = Hq // Hkv
                toks = 128 // g
                pairs = B * Hkv * -(--(-new // toks) // 2)
                for Lk in (64, 4096, 32768, 131072, 1 << 20):
                    need = fl.attn_fwd_paged_fp8_workspace_bytes(B, B * new, new, Hq, Hkv, Lk, d)
                    rows = pairs % 148 * 2 * toks * g
                    assert 32 <= need <= 32 + rows * 32 * (d + 1) * 4, (B, new, Hq, Hkv, Lk)
                    assert rows == 0 or (need - 32) % (rows * (d + 1) * 4) == 0
    # as a caller meets it: what was 1.4, 2.2, 3.1, 3.8 and 52 GB by all rows
    for B, new, Hq, Lk, most in ((1, 4800, 32, 131072, 20), (16, 2048, 32, 32768, 56), (3, 1984, 32, 32768, 18), (4, 8192, 32, 131072, 89),
                                 (3, 8192, 128, 131072, 18)):
        assert fl.attn_fwd_paged_fp8_workspace_bytes(B, B * new, new, Hq, 8, Lk, 128) <= most << 20


def test_reference_rounding():
    """The reference's e4m3 against torch's conversion, on every value and every midpoint."""
    v = ref.TABLE[:127]
    assert torch.equal(ref.round_e4m3(v), v)
    mid = (v[1:] + v[:-1]) / 2
    for x in (mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)):
        x = torch.cat([x, -x])
        assert torch.equal(ref.round_e4m3(x), x.float().to(torch.float8_e4m3fn).double())


def test_reference_append_errors():
    """Written rows are off by at most half a step of their scale, through any number of growing scales."""
    g = torch.Generator().manual_seed(3)
    P, H, d = 16, 2, 64
    values, scales = torch.zeros(3, P, H, d, dtype=torch.float64), torch.ones(3, H, dtype=torch.float64)
    x = torch.randn(P, H, d, generator=g, dtype=torch.float64) * torch.exp(torch.linspace(-6, 6, P, dtype=torch.float64))[:, None, None]
    grown = 0.0
    for t in range(P):
        ref.append(x[t:t + 1], [P + t], values, scales)
        grown = grown + 2.0 ** -10 * scales[1]
    err = (values[1] * scales[1][None, :, None] - x).abs()
    # one rounding when written, and at most one subnormal rounding per growth of the scale
    assert bool((err <= 2.0 ** -4 * x.abs() + grown[None, :, None]).all())
    assert torch.equal(torch.frexp(scales[1])[0], torch.full((H,), 0.5, dtype=torch.float64))  # powers of two
    assert bool((x.abs().amax((0, 2)) <= 448 * scales[1]).all())


def test_reference_plan_closed_form():
    slots, cu, lens, counts, table = ref.plan([0, 16, 5], [17, 1, 3], [7, 8, 9, 4], [[-1, -1], [3, -1], [6, -1]], 16, 24)
    assert slots == [7 * 16 + i for i in range(16)] + [8 * 16] + [9 * 16] + [6 * 16 + 5, 6 * 16 + 6, 6 * 16 + 7] + [-1] * 3
    assert cu == [0, 17, 18, 21] and lens == [17, 17, 8] and counts == [21, 3]
    assert table == [[7, 8], [3, 9], [6, -1]]
