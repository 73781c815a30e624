"""The paged 8-bit KV cache on the GPU (plan, append, decode, multi-token
attention) against the plain 64-bit implementations of tests/_paged_ref.py."""
import math
import threading

import pytest
import torch

from tests import _paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fl():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from io_aware_exact_34_b200 import build
    build.build()
    from io_aware_exact_34_b200 import fattn
    return fattn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(lens, page, width, pages, g):
    """Distinct random pages for every sequence's length; -1 elsewhere."""
    order = torch.randperm(pages, generator=g).tolist()
    out = []
    for n in lens:
        k = -(-n // page)
        out.append([order.pop() for _ in range(k)] + [-1] * (width - k))
    return out


def _cache(pages, page, hkv, d, g, spread=2):
    """Random codes (no NaN) and power-of-two scales 2^-7 * 2^[-spread, spread]."""
    def codes():
        c = torch.randint(0, 256, (pages, page, hkv, d), generator=g, dtype=torch.int32)
        x = torch.randn(c.shape, generator=g) * 90.0  # the values a quantizer leaves
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    def scales():
        return torch.exp2(torch.randint(-7 - spread, -7 + spread + 1, (pages, hkv), generator=g).float())
    return codes(), codes(), scales(), scales()


# ---------------------------------------------------------------- plan
PLAN_CASES = {
    "one": ([0], [1], 16, 2, 4, 1),
    "decode": ([31, 32, 33, 0, 15], [1] * 5, 16, 4, 8, 5),
    "prompts": ([0, 100, 64, 7], [300, 0, 129, 1000], 64, 17, 40, 1500),
    "short capacity": ([5, 9], [40, 40], 16, 8, 9, 50),
    "short free list": ([5, 9, 0], [40, 40, 40], 16, 8, 4, 130),
    "no free list": ([5, 16], [3, 3], 16, 8, 0, 8),
    "short table": ([5, 9], [100, 3], 32, 2, 9, 110),
    "negative": ([-3, 20], [4, -5], 16, 4, 3, 9),
    "nothing": ([3, 4], [0, 0], 16, 4, 3, 2),
}


@pytest.mark.parametrize("name", PLAN_CASES)
def test_plan_matches_reference(fl, name):
    lens, new, page, width, nfree, room = PLAN_CASES[name]
    g = torch.Generator().manual_seed(len(name))
    table = _table([max(0, min(x, width * page)) for x in lens], page, width, 64, g)
    free = [100 + int(i) for i in torch.randperm(nfree, generator=g)]
    dev = _i32(table)
    slots, cu, out, counts = fl.attn_paged_plan(_i32(lens), _i32(new), _i32(free), dev, page, room)
    e_slots, e_cu, e_out, e_counts, e_table = ref.plan(lens, new, free, table, page, room)
    assert slots.tolist() == e_slots and cu.tolist() == e_cu and out.tolist() == e_out
    assert counts.tolist() == e_counts and dev.tolist() == e_table


@pytest.mark.parametrize("B,longest,new,page", [(1, 1, 20000, 16), (257, 500, 90, 32), (4096, 64, 1, 16), (16384, 300, 3, 128)])
def test_plan_sizes(fl, B, longest, new, page):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    adds = torch.randint(0, new + 1, (B,), generator=g).tolist()
    adds[-1] = new
    width = -(-(longest + new) // page)
    held = sum(-(-x // page) for x in lens)
    table = _table(lens, page, width, held, g)
    need = sum(-(-(x + a) // page) - -(-x // page) for x, a in zip(lens, adds))
    free = (held + torch.randperm(need, generator=g)).tolist()
    room = sum(adds) + 3
    dev = _i32(table)
    slots, cu, out, counts = fl.attn_paged_plan(_i32(lens), _i32(adds), _i32(free), dev, page, room)
    e = ref.plan(lens, adds, free, table, page, room)
    for x, y in zip((slots, cu, out, counts, dev), e):
        assert x.tolist() == y


def test_plan_saturates(fl):
    """Sums beyond 31 bits are written as 2^31 - 1 and reach no memory."""
    lens, new = [2 ** 31 - 5, 2 ** 31 - 1, 3], [2 ** 31 - 1, 7, 2]
    table = _i32([[0, 1]] * 3)
    slots, cu, out, counts = fl.attn_paged_plan(_i32(lens), _i32(new), _i32([5, 6]), table, 16, 64)
    assert slots.tolist() == [-1] * 64 and cu.tolist() == [0] + [2 ** 31 - 1] * 3
    assert out.tolist() == [2 ** 31 - 1, 2 ** 31 - 1, 5] and counts[0] == 2 ** 31 - 1
    assert table.tolist() == [[0, 1]] * 3


def test_plan_results_stand_alone(fl):
    """The results of one call can be changed, kept and fed back one by one."""
    for B in (1, 31, 32, 33, 500):
        table = _i32([[b] for b in range(B)])
        got = fl.attn_paged_plan(_i32([1] * B), _i32([2] * B), _i32([]), table, 16, 2 * B)
        want = [t.tolist() for t in got]
        assert want[1] == list(range(0, 2 * B + 1, 2)) and want[2] == [3] * B and want[3] == [2 * B, 0]
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in got)
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
        assert all(t.is_contiguous() and t.data_ptr() % 128 == 0 for t in got)
        for i, t in enumerate(got):
            t.fill_(-9)
            assert [x.tolist() for x in got[i + 1:]] == want[i + 1:]
        got = fl.attn_paged_plan(_i32([1] * B), _i32([2] * B), _i32([]), table, 16, 2 * B)
        again = fl.attn_paged_plan(got[2], _i32([1] * B), _i32([]), table, 16, B)
        assert again[2].tolist() == [4] * B and got[2].tolist() == [3] * B


# ---------------------------------------------------------------- append
def _append_and_check(fl, x, slots, cache, page):
    """x: bf16 (k, v) on the GPU, any token stride; cache: CPU codes and scales."""
    kc, vc, ks, vs = [t.cuda() for t in cache]
    fl.attn_append_paged_fp8(x[0], x[1], torch.tensor(slots, dtype=torch.int64, device="cuda"), kc, vc, ks, vs)
    for t, c, s, c0, s0 in ((x[0], kc, ks, cache[0], cache[2]), (x[1], vc, vs, cache[1], cache[3])):
        values, scales = ref.value(c0), s0.double()
        ref.append(t.double().cpu(), slots, values, scales)
        assert torch.equal(s.double().cpu(), scales)
        assert torch.equal(ref.value(c.cpu()).nan_to_num(1e9), values.nan_to_num(1e9))
    return kc, vc, ks, vs


@pytest.mark.parametrize("lens,new,page,hkv,d", [
    ([0], [1], 16, 1, 128), ([15, 16, 17, 0, 3], [1] * 5, 16, 8, 128), ([3, 0, 40], [50, 16, 9], 16, 2, 64),
    ([0, 100, 31, 64], [200, 1, 90, 64], 64, 3, 128), ([250, 0], [300, 513], 256, 2, 128), ([1, 0, 129], [700, 256, 1], 256, 1, 64),
    ([7, 8], [33, 1], 32, 5, 64), ([100], [1000], 128, 4, 128), ([0], [1500], 1024, 1, 128),
])
def test_append_matches_reference(fl, lens, new, page, hkv, d):
    g = torch.Generator().manual_seed(sum(lens) + page)
    full = [a + b for a, b in zip(lens, new)]
    width, pages = max(-(-x // page) for x in full), sum(-(-x // page) for x in full) + 2
    table = _table(full, page, width, pages, g)
    slots = [table[b][p // page] * page + p % page for b in range(len(lens)) for p in range(lens[b], full[b])]
    cache = _cache(pages, page, hkv, d, g)
    x = torch.randn(len(slots), 2, hkv, d, generator=g) * torch.exp(2 * torch.randn(len(slots), 1, 1, 1, generator=g))
    x = x.to(torch.bfloat16).cuda()  # K and V interleaved: token stride 2 * hkv * d
    _append_and_check(fl, (x[:, 0], x[:, 1]), slots, cache, page)
    _append_and_check(fl, (x[:, 0].contiguous(), x[:, 1].contiguous()), slots, cache, page)


def test_append_skips_and_duplicates(fl):
    """Slots outside the pool are skipped; one named again in a stretch keeps the later token."""
    g = torch.Generator().manual_seed(1)
    cache = _cache(6, 16, 2, 128, g)
    slots = [-1, 5 * 16 + 3, 5 * 16 + 4, 96, -7, 16, 17, 17, 17, 18, 10 ** 12, 3 * 16 + 15, 40, 40]
    x = torch.randn(len(slots), 2, 2, 128, generator=g).to(torch.bfloat16).cuda()
    _append_and_check(fl, (x[:, 0], x[:, 1]), slots, cache, 16)
    slots = [20] * 70  # longer than a page, one row
    x = torch.randn(len(slots), 2, 2, 128, generator=g).to(torch.bfloat16).cuda()
    _append_and_check(fl, (x[:, 0], x[:, 1]), slots, cache, 16)


@pytest.mark.parametrize("slots", [[20], [20, 21], [16, 17, 17, 18, 31]])
def test_append_many_tokens_of_few_slots(fl, slots):
    """A long stretch over a few slots (a batch padded with one spare slot) takes time linear in its tokens."""
    g = torch.Generator().manual_seed(6)
    cache = _cache(3, 16, 1, 64, g)
    n = 60000
    slots = sorted(slots * (n // len(slots))) if len(slots) > 2 else slots * (n // len(slots))
    x = torch.randn(len(slots), 2, 1, 64, generator=g).to(torch.bfloat16).cuda()
    _append_and_check(fl, (x[:, 0], x[:, 1]), slots, cache, 16)
    dev = [t.cuda() for t in cache]
    at = torch.tensor(slots, dtype=torch.int64, device="cuda")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    fl.attn_append_paged_fp8(x[:, 0], x[:, 1], at, *dev)
    end.record()
    torch.cuda.synchronize()
    # n / 4 rows a lane at a few loads each; a look through the whole rest of the stretch for each would be 4e8 loads a lane
    assert begin.elapsed_time(end) < 500.0


def test_append_extremes(fl):
    """Zeros, subnormals, the largest bf16, exact scale borders, infinities and NaN."""
    g = torch.Generator().manual_seed(2)
    H, d = 2, 64
    rows = [torch.zeros(H, d), torch.full((H, d), 1e-39), torch.full((H, d), 3.3895e38), torch.full((H, d), 448.0 * 2.0 ** -9),
            torch.full((H, d), 450.0 * 2.0 ** -9), torch.full((H, d), -1.75), torch.randn(H, d, generator=g) * 1e-30]
    bad = torch.randn(H, d, generator=g)
    bad[0, 3], bad[0, 5], bad[1, 7] = math.inf, -math.inf, math.nan
    rows += [bad, torch.full((H, d), math.nan)]
    for i, r in enumerate(rows):
        cache = _cache(3, 16, H, d, g)
        x = r[None].to(torch.bfloat16).cuda()
        for slot in (16, 16 + 5):  # a fresh page, and one with rows before
            _append_and_check(fl, (x, x), [slot], cache, 16)
    # all of them one after the other into one page: the scale grows over the whole range
    cache = _cache(3, 16, H, d, g)
    for i, r in enumerate(rows):
        x = r[None].to(torch.bfloat16).cuda()
        kc, vc, ks, vs = _append_and_check(fl, (x, x), [32 + i], cache, 16)
        cache = (kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu())


def test_append_leaves_the_rest(fl):
    """Other pages, other heads' scales and rows behind the new ones keep their bytes."""
    g = torch.Generator().manual_seed(4)
    cache = _cache(5, 32, 3, 128, g)
    kc, vc, ks, vs = [t.cuda() for t in cache]
    x = (torch.randn(4, 3, 128, generator=g) * 100).to(torch.bfloat16).cuda()
    fl.attn_append_paged_fp8(x, x, torch.arange(2 * 32 + 8, 2 * 32 + 12, device="cuda"), kc, vc, ks, vs)
    for new, old in ((kc, cache[0]), (vc, cache[1])):
        new = new.cpu()
        assert torch.equal(new[[0, 1, 3, 4]], old[[0, 1, 3, 4]]) and torch.equal(new[2, 12:], old[2, 12:])
        assert not torch.equal(new[2, 8:12], old[2, 8:12])
    for new, old in ((ks, cache[2]), (vs, cache[3])):
        assert torch.equal(new.cpu()[[0, 1, 3, 4]], old[[0, 1, 3, 4]])


def test_append_rejects(fl):
    g = torch.Generator().manual_seed(5)
    kc, vc, ks, vs = [t.cuda() for t in _cache(3, 16, 2, 64, g)]
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    for bad in ((x[:1], x), (x.transpose(1, 2).contiguous().transpose(1, 2), x), (x.half(), x), (x.cpu(), x)):
        with pytest.raises((ValueError, TypeError), match="k:"):
            fl.attn_append_paged_fp8(*bad, slots, kc, vc, ks, vs)
    with pytest.raises(ValueError, match="v_scales:"):
        fl.attn_append_paged_fp8(x, x, slots, kc, vc, ks, vs[:2])
    with pytest.raises(ValueError, match="v_pages:"):
        fl.attn_append_paged_fp8(x, x, slots, kc, vc[:, :8], ks, vs)
    with pytest.raises(ValueError, match="slot_map:"):
        fl.attn_append_paged_fp8(x, x, slots.int(), kc, vc, ks, vs)
    with pytest.raises(fl.FattnError):
        fl.attn_append_paged_fp8(x, x, slots, kc, kc, ks, vs)
    odd = torch.zeros(2, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, :128].view(2, 2, 64)
    with pytest.raises(fl.FattnError):
        fl.attn_append_paged_fp8(odd, x, slots, kc, vc, ks, vs)


# ---------------------------------------------------------------- attention
def _check_rows(o, lse, exp, d, length, label=""):
    """o [n, Hq, d], lse [n, Hq] of the GPU against ref.attention's answer."""
    eo, el, w, dots = exp
    o, lse = o.double().cpu(), lse.double().cpu()
    empty = el == -math.inf
    assert torch.equal(lse == -math.inf, empty), label
    assert bool((o[empty] == 0).all()), label
    bad = eo.isnan()
    assert torch.equal(o.isnan(), bad), label
    to, tl = ref.tolerances(eo, w, dots, d, max(1, length))
    far = torch.where(bad, 0.0, (o - eo).abs() - to)
    assert float(far.max()) <= 0.0, f"{label}: O off by {float(far.max()):.3e} more than its bound"
    fine = ~empty & ~el.isnan()
    if fine.any():
        far = ((lse - el).abs() - tl)[fine]
        assert float(far.max()) <= 0.0, f"{label}: LSE off by {float(far.max()):.3e} more than its bound"


def _decode_case(fl, lens, page, hq, hkv, d, seed, left=-1, splits=0, spread=2, spoil=True, q_gain=1.0):
    g = torch.Generator().manual_seed(seed)
    width = max(1, max(-(-x // page) for x in lens)) + 1
    pages = sum(-(-x // page) for x in lens) + 2
    table = _table(lens, page, width, pages, g)
    kc, vc, ks, vs = _cache(pages, page, hkv, d, g, spread)
    q = (torch.randn(len(lens), hq, 1, d, generator=g) * q_gain).to(torch.bfloat16)
    if spoil:
        # rows behind the lengths and pages no table names: NaN codes and NaN scales
        named = torch.zeros(pages, dtype=torch.bool)
        for b, n in enumerate(lens):
            for p in range(-(-n // page)):
                named[table[b][p]] = True
                kc[table[b][p], max(0, n - p * page):] = 0x7F
                vc[table[b][p], max(0, n - p * page):] = 0xFF
        for t in (ks, vs):
            t[~named] = math.nan
        for t in (kc, vc):
            t[~named] = 0x7F
    o, lse = fl.attn_decode_paged_fp8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), _i32(table), _i32(lens),
                                      window_left=left, num_splits=splits)
    kv, vv = ref.value(kc), ref.value(vc)
    for b, n in enumerate(lens):
        exp = ref.attention(q[b, :, 0].double()[None], ref.gather(kv, ks.double(), table[b], n), ref.gather(vv, vs.double(), table[b], n),
                            float(torch.tensor(d ** -0.5, dtype=torch.float32)), left=left)
        _check_rows(o[b, :, 0][None], lse[b][None], exp, d, n, f"sequence {b} of {n} keys")


@pytest.mark.parametrize("lens,page,hq,hkv,d,left,splits", [
    ([1], 16, 1, 1, 128, -1, 0), ([0, 1, 15, 16, 17, 63, 64, 65], 16, 4, 1, 128, -1, 0), ([0, 0], 16, 2, 2, 64, -1, 0),
    ([300, 5, 1000], 16, 8, 8, 128, -1, 1), ([300, 5, 1000], 16, 8, 8, 64, -1, 3), ([4097, 2], 64, 32, 8, 128, -1, 0),
    ([777, 1555], 256, 16, 2, 128, -1, 7), ([777, 1555], 32, 16, 1, 64, -1, 0), ([130, 1029], 128, 12, 4, 128, -1, 0),
    ([500], 16, 10, 2, 64, -1, 2), ([999, 48], 16, 32, 1, 128, -1, 0), ([333], 16, 71, 1, 64, -1, 0), ([40, 200], 16, 128, 1, 128, -1, 0),
    ([1000, 3, 129, 0], 16, 8, 2, 128, 100, 0), ([1000, 128], 64, 8, 8, 64, 0, 0), ([2000, 77], 32, 16, 16, 128, 1023, 4),
    ([1 << 14], 16, 8, 2, 128, -1, 64),
])
def test_decode_matches_reference(fl, lens, page, hq, hkv, d, left, splits):
    _decode_case(fl, lens, page, hq, hkv, d, seed=sum(lens) + hq, left=left, splits=splits)


@pytest.mark.parametrize("splits,left", [(65, -1), (100, -1), (128, -1), (128, 20000), (200, -1)])
def test_decode_more_than_64_splits(fl, splits, left):
    """As many parts of a sequence as num_splits asks for, beside sequences that have fewer of them."""
    lens = [33280, 700, 24001, 0, 16640]
    _decode_case(fl, lens, 16, 4, 2, 128, seed=splits, left=left, splits=splits, q_gain=8.0)
    _decode_case(fl, lens, 64, 3, 1, 64, seed=splits + 1, left=left, splits=splits, q_gain=8.0)


@pytest.mark.parametrize("spread,q_gain", [(20, 1.0), (5, 30.0), (0, 1e-20), (2, 0.0)])
def test_decode_ranges(fl, spread, q_gain):
    """Page scales far apart, sharp and flat softmax rows."""
    _decode_case(fl, [700, 65, 2100], 16, 8, 2, 128, seed=9, spread=spread, q_gain=q_gain)
    _decode_case(fl, [700, 65, 2100], 32, 16, 1, 64, seed=9, spread=spread, q_gain=q_gain)


def test_decode_not_power_of_two_scales(fl):
    g = torch.Generator().manual_seed(11)
    lens, page = [100, 515], 16
    pages = sum(-(-x // page) for x in lens)
    table = _table(lens, page, 33, pages, g)
    kc, vc, _, _ = _cache(pages, page, 2, 128, g)
    ks, vs = [torch.rand(pages, 2, generator=g) * 0.02 + 1e-4 for _ in range(2)]
    q = torch.randn(2, 8, 1, 128, generator=g).to(torch.bfloat16)
    o, lse = fl.attn_decode_paged_fp8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), _i32(table), _i32(lens), scale=0.25)
    for b, n in enumerate(lens):
        exp = ref.attention(q[b, :, 0].double()[None], ref.gather(ref.value(kc), ks.double(), table[b], n),
                            ref.gather(ref.value(vc), vs.double(), table[b], n), 0.25)
        _check_rows(o[b, :, 0][None], lse[b][None], exp, 128, n)


def test_decode_visible_nan(fl):
    """A NaN in a visible K row spoils its head's rows; one in V only its column; a NaN query only itself."""
    g = torch.Generator().manual_seed(12)
    lens, page = [100, 200], 16
    pages = sum(-(-x // page) for x in lens)
    table = _table(lens, page, 14, pages, g)
    kc, vc, ks, vs = _cache(pages, page, 2, 128, g)
    kc[table[0][2], 3, 1, 9] = 0x7F
    vc[table[1][4], 7, 0, 77] = 0xFF
    q = torch.randn(2, 8, 1, 128, generator=g).to(torch.bfloat16)
    q[1, 6, 0, 5] = math.nan
    for splits in (0, 1, 2):
        o, lse = fl.attn_decode_paged_fp8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), _i32(table), _i32(lens), num_splits=splits)
        want = torch.zeros(2, 8, 1, 128, dtype=torch.bool)
        want[0, 4:] = True
        want[1, :4, 0, 77] = True
        want[1, 6] = True
        assert torch.equal(o.isnan().cpu(), want)
        assert torch.equal(lse.isnan().cpu(), want.all(-1)[..., 0])


@pytest.mark.parametrize("new", [1, 40])
def test_queries_that_are_not_finite(fl, new):
    """An infinity or a NaN in a query row spoils that row and no other, in short and in long runs."""
    g = torch.Generator().manual_seed(16)
    kc, vc, ks, vs = [t.cuda() for t in _cache(8, 16, 2, 128, g)]
    q = torch.randn(new, 4, 128, generator=g).to(torch.bfloat16)
    clean = q.clone()
    q[0, 1, 3], q[new - 1, 2, 100], q[new // 2, 0, 64] = math.inf, -math.inf, math.nan
    bad = ~q.isfinite().all(-1)
    a = fl.attn_fwd_paged_fp8(q.cuda(), kc, vc, ks, vs, _i32([list(range(8))]), _i32([100]), _i32([0, new]), new, causal=True)
    b = fl.attn_fwd_paged_fp8(clean.cuda(), kc, vc, ks, vs, _i32([list(range(8))]), _i32([100]), _i32([0, new]), new, causal=True)
    assert torch.equal(a[0].isnan().cpu(), bad[..., None].expand(q.shape)) and torch.equal(a[1].isnan().cpu(), bad.T)
    assert torch.equal(a[0].cpu()[~bad], b[0].cpu()[~bad]) and torch.equal(a[1].T.cpu()[~bad], b[1].T.cpu()[~bad])


def test_decode_bad_tables_and_lengths(fl):
    """Table entries outside the pool are clamped, lengths beyond the table too: same as with the clamped ones."""
    g = torch.Generator().manual_seed(13)
    kc, vc, ks, vs = [t.cuda() for t in _cache(6, 16, 2, 64, g)]
    q = torch.randn(2, 4, 1, 64, generator=g).to(torch.bfloat16).cuda()
    a = fl.attn_decode_paged_fp8(q, kc, vc, ks, vs, _i32([[-5, 2, 99], [3, 1 << 30, 0]]), _i32([1000, -4]))
    b = fl.attn_decode_paged_fp8(q, kc, vc, ks, vs, _i32([[0, 2, 5], [3, 5, 0]]), _i32([48, 0]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert bool((a[0][1] == 0).all()) and bool((a[1][1] == -math.inf).all())


def test_decode_far_offsets(fl):
    """Pages whose byte offsets pass 32 bits."""
    hkv, d, page = 8, 128, 256
    pages = (5 << 30) // (page * hkv * d)
    kc = torch.empty(pages, page, hkv, d, dtype=torch.uint8, device="cuda")
    vc = torch.empty_like(kc)
    ks, vs = torch.empty(pages, hkv, device="cuda"), torch.empty(pages, hkv, device="cuda")
    g = torch.Generator().manual_seed(14)
    small = _cache(3, page, hkv, d, g)
    at = torch.tensor([pages - 1, 3, pages - 2], device="cuda")
    for big, t in zip((kc, vc, ks, vs), small):
        big[at] = t.cuda()
    q = torch.randn(1, 32, 1, d, generator=g).to(torch.bfloat16).cuda()
    a = fl.attn_decode_paged_fp8(q, kc, vc, ks, vs, at.int()[None], _i32([700]))
    b = fl.attn_decode_paged_fp8(q, *[t.cuda() for t in small], _i32([[0, 1, 2]]), _i32([700]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = torch.randn(2, hkv, d, generator=g).to(torch.bfloat16).cuda()
    fl.attn_append_paged_fp8(x, x, torch.tensor([pages * page - 2, pages * page - 1], device="cuda"), kc, vc, ks, vs)
    want = [t.cuda() for t in small]
    fl.attn_append_paged_fp8(x, x, torch.tensor([254, 255], device="cuda"), *want)
    assert torch.equal(kc[-1], want[0][0]) and torch.equal(vs[-1], want[3][0])


def test_decode_rejects(fl):
    g = torch.Generator().manual_seed(15)
    kc, vc, ks, vs = [t.cuda() for t in _cache(3, 16, 2, 64, g)]
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    bt, lens = _i32([[0, 1], [2, 0]]), _i32([20, 3])
    call = lambda **kw: fl.attn_decode_paged_fp8(**{**dict(q=q, k_pages=kc, v_pages=vc, k_scales=ks, v_scales=vs, block_table=bt, seqlens_k=lens), **kw})  # noqa: E731
    call()
    for bad, match in ((dict(q=q[:, :3].contiguous()), "k_pages:"), (dict(q=q.repeat(1, 1, 2, 1)), "one query"), (dict(q=q[..., :32].contiguous()), "k_pages:"),
                       (dict(block_table=bt[:1]), "block_table:"), (dict(seqlens_k=lens[:1]), "seqlens_k:"), (dict(k_scales=ks[:, :1].contiguous()), "k_scales:"),
                       (dict(v_pages=vc.float()), "v_pages:"), (dict(o=q[:1]), "o:"), (dict(lse=torch.zeros(2, 3, device="cuda")), "lse:"),
                       (dict(workspace=torch.zeros(8)), "workspace:")):
        with pytest.raises(ValueError, match=match):
            call(**bad)
    for bad in (dict(num_splits=-1), dict(num_splits=33), dict(scale=-1.0), dict(num_splits=2, workspace=torch.zeros(16, device="cuda"))):
        with pytest.raises(fl.FattnError):
            call(**bad)


# ---------------------------------------------------------------- several tokens
def _fwd_case(fl, lens, new, page, hq, hkv, d, seed, causal=True, left=-1, right=-1, behind=0, most=None, spread=2, nan_v=None):
    g = torch.Generator().manual_seed(seed)
    width = max(1, max(-(-x // page) for x in lens)) + 1
    pages = sum(-(-x // page) for x in lens) + 1
    table = _table(lens, page, width, pages, g)
    kc, vc, ks, vs = _cache(pages, page, hkv, d, g, spread)
    for b, n in enumerate(lens):
        if n % page:
            kc[table[b][n // page], n % page:] = 0x7F
            vc[table[b][n // page], n % page:] = 0x7F
    for b, pos, h, e in nan_v or []:
        vc[table[b][pos // page], pos % page, h, e] = 0x7F
    total = sum(new) + behind
    q = torch.randn(total, hq, d, generator=g).to(torch.bfloat16)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    o = torch.full((total, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hq, total), 7.0, device="cuda")
    most = max(1, max(new)) if most is None else most
    fl.attn_fwd_paged_fp8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), _i32(table), _i32(lens), _i32(cu), most, o=o, lse=lse,
                          causal=causal, window_left=left, window_right=right)
    kv, vv = ref.value(kc), ref.value(vc)
    for b, n in enumerate(new):
        if n == 0:
            continue
        exp = ref.attention(q[cu[b]:cu[b + 1]].double(), ref.gather(kv, ks.double(), table[b], lens[b]),
                            ref.gather(vv, vs.double(), table[b], lens[b]), float(torch.tensor(d ** -0.5, dtype=torch.float32)),
                            causal=causal, left=left, right=right)
        m = min(n, most)
        _check_rows(o[cu[b]:cu[b] + m], lse[:, cu[b]:cu[b] + m].T, [t[:m] for t in exp], d, lens[b], f"sequence {b}: {n} of {lens[b]}")
        assert bool((o[cu[b] + m:cu[b + 1]] == 7).all()) and bool((lse[:, cu[b] + m:cu[b + 1]] == 7).all())
    assert bool((o[sum(new):] == 7).all()) and bool((lse[:, sum(new):] == 7).all())


FWD_CASES = [
    # lens, new, page, hq, hkv, d, mask
    ([1], [1], 16, 1, 1, 128, {}), ([40, 5, 0, 17], [3, 5, 0, 1], 16, 4, 2, 128, {}), ([300, 129], [2, 129], 16, 8, 8, 64, {}),
    ([1000, 33, 512], [5, 5, 4], 16, 32, 8, 128, {}), ([700, 64], [300, 64], 64, 8, 1, 128, {}), ([257, 1111], [257, 140], 32, 6, 2, 64, {}),
    ([500], [260], 256, 5, 1, 128, {}), ([300], [37], 16, 71, 1, 64, {}), ([140], [9], 16, 128, 1, 128, {}),
    ([900, 100], [400, 100], 16, 4, 4, 128, dict(left=64)), ([900, 100], [130, 1], 64, 8, 2, 64, dict(left=0)),
    ([300, 50], [200, 50], 16, 4, 2, 128, dict(causal=False)), ([300, 50], [200, 50], 16, 4, 2, 64, dict(causal=False, left=30, right=20)),
    ([20, 0, 3], [50, 7, 3], 16, 4, 2, 128, {}), ([20, 5], [50, 9], 16, 2, 1, 64, dict(left=3)), ([5], [300], 16, 4, 1, 128, dict(causal=False, right=2)),
    ([600, 80], [256, 80], 128, 16, 4, 128, dict(behind=5)), ([600, 80], [256, 20], 16, 4, 2, 128, dict(most=33)),
    ([900], [300], 16, 4, 2, 128, dict(spread=20)),
    # few rows: sequences without keys, rows behind the last sequence, splits
    ([0, 30, 0], [2, 3, 0], 16, 4, 2, 128, dict(behind=4)), ([5000, 3], [4, 2], 16, 8, 2, 128, {}), ([9000], [3], 64, 4, 1, 64, dict(left=5000)),
    ([700, 20], [6, 6], 32, 4, 1, 128, dict(most=4)),
    # keys in several parts, some of them without a key for some rows
    ([3000, 700, 5], [100, 64, 5], 16, 8, 2, 128, {}), ([2500], [40], 64, 8, 1, 64, dict(left=900)),
    ([2100, 1300], [70, 70], 32, 4, 4, 128, dict(causal=False)), ([2600], [33], 16, 16, 4, 64, dict(causal=False, left=700, right=300)),
    ([4200], [1400], 256, 2, 1, 128, dict(left=300)), ([1030, 40], [1030, 600], 128, 2, 2, 64, {}),
]


@pytest.mark.parametrize("lens,new,page,hq,hkv,d,kw", FWD_CASES)
def test_fwd_matches_reference(fl, lens, new, page, hq, hkv, d, kw):
    _fwd_case(fl, lens, new, page, hq, hkv, d, seed=sum(lens) + hq, **kw)


@pytest.mark.parametrize("hq,hkv,d,new", [(4, 2, 128, 5), (4, 1, 64, 3), (4, 2, 128, 200), (8, 2, 64, 150)])
def test_fwd_nan_values_spare_rows_that_do_not_see_them(fl, hq, hkv, d, new):
    """A NaN in V reaches its column in the rows that see its key, and no other row."""
    _fwd_case(fl, [300, 220], [new, 1], 16, hq, hkv, d, seed=3, nan_v=[(0, 298, hkv - 1, 5), (0, 300 - new, 0, 0), (1, 219, 0, d - 1)])
    _fwd_case(fl, [300], [new], 16, hq, hkv, d, seed=4, left=40, nan_v=[(0, 290, 0, 1), (0, 300 - new - 20, hkv - 1, 2)])


def test_fwd_nan_values_in_parts(fl):
    """The same where the keys are cut into parts."""
    _fwd_case(fl, [2900], [90], 16, 4, 2, 128, seed=5, nan_v=[(0, 2890, 0, 5), (0, 2830, 1, 0), (0, 2899, 1, 127)])
    _fwd_case(fl, [2900], [90], 32, 4, 1, 64, seed=6, left=1500, nan_v=[(0, 2895, 0, 5), (0, 1330, 0, 0), (0, 1400, 0, 63)])


@pytest.mark.parametrize("lens,new,page,hq,hkv,d,left", [
    ([5000, 900], [1300, 60], 64, 32, 8, 128, -1), ([3000], [2500], 16, 16, 16, 64, -1), ([3000], [2500], 16, 16, 16, 64, 700),
    ([4000], [401], 128, 71, 1, 128, -1), ([16000, 40], [600, 3], 256, 8, 8, 128, -1),
])
def test_fwd_whole_and_cut_pairs(fl, lens, new, page, hq, hkv, d, left):
    """More pairs of row tiles than one round holds, the last round's cut into parts, in a workspace of the size asked for
    and no byte more: rows of both kinds, and the same bits as with the library's own workspace."""
    g = torch.Generator().manual_seed(sum(new) + hq)
    width = -(-max(lens) // page) + 1
    pages = sum(-(-x // page) for x in lens) + 1
    table = _table(lens, page, width, pages, g)
    cache = _cache(pages, page, hkv, d, g)
    q = torch.randn(sum(new), hq, d, generator=g).to(torch.bfloat16)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    args = (q.cuda(), *[t.cuda() for t in cache], _i32(table), _i32(lens), _i32(cu), max(new))
    need = fl.attn_fwd_paged_fp8_workspace_bytes(len(lens), sum(new), max(new), hq, hkv, width * page, d)
    buf = torch.full((need + 128,), 0x5A, dtype=torch.uint8, device="cuda")
    o, lse = fl.attn_fwd_paged_fp8(*args, causal=True, window_left=left, workspace=buf[64:64 + need])
    assert bool((buf[:64] == 0x5A).all()) and bool((buf[64 + need:] == 0x5A).all())
    o2, lse2 = fl.attn_fwd_paged_fp8(*args, causal=True, window_left=left)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    kv, vv = ref.value(cache[0]), ref.value(cache[1])
    for b, n in enumerate(new):
        k, v = ref.gather(kv, cache[2].double(), table[b], lens[b]), ref.gather(vv, cache[3].double(), table[b], lens[b])
        for i in sorted({0, 1, n - 1, n // 2} | set(torch.randint(0, n, (12,), generator=g).tolist())):
            at, seen = cu[b] + i, lens[b] - n + i + 1
            exp = ref.attention(q[at][None].double(), k[:seen], v[:seen], float(torch.tensor(d ** -0.5, dtype=torch.float32)), left=left)
            _check_rows(o[at][None], lse[:, at][None], exp, d, seen, f"sequence {b}, token {i}")


def test_fwd_one_token_is_decode(fl):
    """One new token per sequence: the rows of attn_decode_paged_fp8, bit for bit when both choose the same splits."""
    g = torch.Generator().manual_seed(21)
    lens, page, hq, hkv, d = [900, 31, 16, 2048], 16, 8, 2, 128
    pages = sum(-(-x // page) for x in lens)
    table = _i32(_table(lens, page, 128, pages, g))
    cache = [t.cuda() for t in _cache(pages, page, hkv, d, g)]
    q = torch.randn(4, hq, 1, d, generator=g).to(torch.bfloat16).cuda()
    o, lse = fl.attn_decode_paged_fp8(q, *cache, table, _i32(lens))
    o2, lse2 = fl.attn_fwd_paged_fp8(q[:, :, 0].contiguous(), *cache, table, _i32(lens), _i32([0, 1, 2, 3, 4]), 1, causal=True)
    assert torch.equal(o[:, :, 0], o2) and torch.equal(lse, lse2.T)


def test_fwd_rejects(fl):
    g = torch.Generator().manual_seed(22)
    kc, vc, ks, vs = [t.cuda() for t in _cache(3, 16, 2, 64, g)]
    q = torch.zeros(6, 4, 64, dtype=torch.bfloat16, device="cuda")
    bt, lens, cu = _i32([[0, 1], [2, 0]]), _i32([20, 3]), _i32([0, 4, 6])
    call = lambda **kw: fl.attn_fwd_paged_fp8(**{**dict(q=q, k_pages=kc, v_pages=vc, k_scales=ks, v_scales=vs, block_table=bt, seqlens_k=lens, cu_seqlens_q=cu, max_seqlen_q=4, causal=True), **kw})  # noqa: E731
    call()
    for bad, match in ((dict(q=q[:, :3].contiguous()), "k_pages:"), (dict(cu_seqlens_q=cu[:2]), "cu_seqlens_q:"), (dict(block_table=bt[:1]), "block_table:"),
                       (dict(o=q[:5]), "o:"), (dict(lse=torch.zeros(6, 4, device="cuda")), "lse:"), (dict(v_scales=ks[:2]), "v_scales:")):
        with pytest.raises(ValueError, match=match):
            call(**bad)
    for bad in (dict(max_seqlen_q=0), dict(scale=0.0)):
        with pytest.raises(fl.FattnError):
            call(**bad)


def test_value_scale_of_nothing(fl):
    """V scales far below every other, and of 0: their rows count as keys and add (next to) nothing."""
    g = torch.Generator().manual_seed(23)
    kc, vc, ks, vs = _cache(4, 16, 1, 128, g)
    q = torch.randn(1, 2, 1, 128, generator=g).to(torch.bfloat16)
    for tiny in (0.0, 2.0 ** -140, 2.0 ** -60):
        small = vs.clone()
        small[1:3] = tiny
        for v in (small, torch.full_like(vs, tiny)):
            exp = ref.attention(q[0, :, 0].double()[None], ref.gather(ref.value(kc), ks.double(), [0, 1, 2, 3], 60),
                                ref.gather(ref.value(vc), v.double(), [0, 1, 2, 3], 60), float(torch.tensor(128 ** -0.5, dtype=torch.float32)))
            args = (kc.cuda(), vc.cuda(), ks.cuda(), v.cuda(), _i32([[0, 1, 2, 3]]), _i32([60]))
            o, lse = fl.attn_decode_paged_fp8(q.cuda(), *args)
            assert bool(((o[:, :, 0].double().cpu() - exp[0]).abs() <= ref.tolerances(*[exp[i] for i in (0, 2, 3)], 128, 60)[0] + 2.0 ** -70).all())
            assert bool(((lse.double().cpu() - exp[1]).abs() <= ref.tolerances(*[exp[i] for i in (0, 2, 3)], 128, 60)[1]).all())


@pytest.mark.parametrize("new", [1, 4, 60])
@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 2), (64, 3, 1)])
def test_value_scales_far_apart(fl, new, d, hq, hkv):
    """Pages with a V scale 2^ratio times that of the others and nothing but zero codes: O is the others' rows alone.

    P is rounded as f16 of p' = 2^7 p vs / m, with m at most the row's largest p vs: by 2^-11 of itself, or by half a
    subnormal step, 2^-25, which is 2^-32 m in p vs.  So beside the other roundings O is off by up to 2^-32 m sum |code|."""
    g = torch.Generator().manual_seed(25)
    pages, page = 12, 16
    L, scale = pages * page - 3, float(torch.tensor(d ** -0.5, dtype=torch.float32))
    kc, vc, ks, _ = _cache(pages, page, hkv, d, g)
    vc[[0, 5]] = 0
    q = torch.randn(new, hq, d, generator=g).to(torch.bfloat16)
    k = ref.gather(ref.value(kc), ks.double(), list(range(pages)), L)
    codes = ref.value(vc).reshape(-1, hkv, d)[:L]
    for ratio in (0, 12, 20, 24, 28, 32, 40, 80):
        vs = torch.full((pages, hkv), 2.0 ** -12)
        vs[[0, 5]] = 2.0 ** (ratio - 12)
        v = ref.gather(ref.value(vc), vs.double(), list(range(pages)), L)
        if new == 1:
            o, lse = fl.attn_decode_paged_fp8(q[:, :, None].cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), _i32([list(range(pages))]), _i32([L]))
            o = o[:, :, 0]
        else:
            o, lse = fl.attn_fwd_paged_fp8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), _i32([list(range(pages))]), _i32([L]), _i32([0, new]), new)
            lse = lse.T
        eo, el, w, dots = ref.attention(q.double(), k, v, scale, causal=False)
        to, tl = ref.tolerances(eo, w, dots, d, L)
        for j in range(hq):
            p = torch.softmax(q[:, j].double() @ k[:, j // (hq // hkv)].T * scale, -1)
            most = (p * vs.double()[torch.arange(L) // page, j // (hq // hkv)]).amax(-1)
            to[:, j] += 1.01 * 2.0 ** -32 * most[:, None] * codes[:, j // (hq // hkv)].abs().sum(0)
        assert bool(((o.double().cpu() - eo).abs() <= to).all()), ratio
        assert bool(((lse.double().cpu() - el).abs() <= tl).all()), ratio
        if ratio <= 20:  # above 2^-21 m the other pages' p vs keep their bits: O is off by its own rounding and theirs
            assert float((o.double().cpu() - eo).norm() / eo.norm()) < 2.0 ** -8, ratio


def test_buffers_given(fl):
    """Outputs and workspaces of the caller's: the same results as with the library's choice."""
    g = torch.Generator().manual_seed(24)
    lens, new, page, hq, hkv, d = [3000, 700], [40, 2], 16, 8, 2, 128
    pages = sum(-(-x // page) for x in lens) + 4
    table = _table(lens, page, 200, pages, g)
    cache = [t.cuda() for t in _cache(pages, page, hkv, d, g)]
    q = torch.randn(2, hq, 1, d, generator=g).to(torch.bfloat16).cuda()
    for S in (0, 1, 3, 12):
        a = fl.attn_decode_paged_fp8(q, *cache, _i32(table), _i32(lens), num_splits=S)
        ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
        o, lse = torch.empty_like(q), torch.empty(2, hq, device="cuda")
        b = fl.attn_decode_paged_fp8(q, *cache, _i32(table), _i32(lens), num_splits=S, o=o, lse=lse, workspace=ws)
        assert b[0] is o and b[1] is lse and torch.equal(a[0], o) and torch.equal(a[1], lse)
    for n in ([40, 2], [3, 2]):
        x = torch.randn(sum(n), hq, d, generator=g).to(torch.bfloat16).cuda()
        cu = _i32([0, n[0], sum(n)])
        a = fl.attn_fwd_paged_fp8(x, *cache, _i32(table), _i32(lens), cu, max(n), causal=True)
        ws = torch.empty(fl.attn_fwd_paged_fp8_workspace_bytes(2, sum(n), max(n), hq, hkv, 200 * page, d), dtype=torch.uint8, device="cuda")
        o, lse = torch.empty_like(x), torch.empty(hq, sum(n), device="cuda")
        b = fl.attn_fwd_paged_fp8(x, *cache, _i32(table), _i32(lens), cu, max(n), o=o, lse=lse, causal=True, workspace=ws)
        assert b[0] is o and b[1] is lse and torch.equal(a[0], o) and torch.equal(a[1], lse)
        with pytest.raises(fl.FattnError):
            fl.attn_fwd_paged_fp8(x, *cache, _i32(table), _i32(lens), cu, max(n), causal=True, workspace=ws[:ws.numel() - 64])
    free, held = _i32([pages - 1, pages - 2, pages - 3]), _i32(lens)
    t1, t2 = _i32(table), _i32(table)
    a = fl.attn_paged_plan(held, _i32(new), free, t1, page, 50)
    bufs = [torch.empty_like(t) for t in a]
    b = fl.attn_paged_plan(held, _i32(new), free, t2, page, 50, *bufs)
    assert torch.equal(t1, t2) and all(x is y and torch.equal(x, z) for x, y, z in zip(b, bufs, a))
    with pytest.raises(fl.FattnError):
        fl.attn_paged_plan(held, _i32(new), free, t2, page, 50, seqlens_out=held)
    for bad in (dict(slot_map=bufs[0][:49]), dict(cu_seqlens=bufs[1].long()), dict(counts=bufs[3][:1])):
        with pytest.raises(ValueError):
            fl.attn_paged_plan(held, _i32(new), free, t2, page, 50, **bad)


def test_arguments_beyond_32_bits(fl):
    """A window wider than 32 bits hold is no window; a size of that kind is refused."""
    g = torch.Generator().manual_seed(28)
    cache = [t.cuda() for t in _cache(8, 16, 2, 128, g)]
    table, lens = _i32([list(range(8))]), _i32([128])
    for new in (1, 5, 40):
        q = torch.randn(new, 4, 128, generator=g).to(torch.bfloat16).cuda()
        args = (q, *cache, table, lens, _i32([0, new]))
        want = fl.attn_fwd_paged_fp8(*args, new)
        for w in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 63 - 1):
            got = fl.attn_fwd_paged_fp8(*args, new, window_left=w, window_right=w)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            if new == 1:
                got = fl.attn_decode_paged_fp8(q[:, :, None], *cache, table, lens, window_left=w)
                assert torch.equal(got[0][:, :, 0], want[0]) and torch.equal(got[1].T, want[1])
        with pytest.raises(ValueError, match="max_seqlen_q"):
            fl.attn_fwd_paged_fp8(*args, 2 ** 32 + new)
    with pytest.raises(ValueError, match="num_splits"):
        fl.attn_decode_paged_fp8(q[:1, :, None], *cache, table, lens, num_splits=2 ** 32 + 1)
    for kw, match in ((dict(page_size=2 ** 32 + 16, max_tokens=4), "page_size"), (dict(page_size=16, max_tokens=2 ** 32 + 4), "max_tokens")):
        with pytest.raises(ValueError, match=match):
            fl.attn_paged_plan(lens, lens, _i32([1]), table.clone(), **kw)


def test_window_over_a_long_table(fl):
    """The library splits what the window leaves, whoever brings the buffers: the same bits."""
    g = torch.Generator().manual_seed(27)
    lens, page, hq, hkv, d, width = [20000, 900], 16, 8, 2, 128, 2500
    pages = sum(-(-x // page) for x in lens)
    table = _i32(_table(lens, page, width, pages, g))
    cache = [t.cuda() for t in _cache(pages, page, hkv, d, g)]
    q = torch.randn(2, hq, 1, d, generator=g).to(torch.bfloat16).cuda()
    for left in (-1, 5000, 40):
        a = fl.attn_decode_paged_fp8(q, *cache, table, _i32(lens), window_left=left)
        o, lse = torch.empty_like(q), torch.empty(2, hq, device="cuda")
        fl.attn_decode_paged_fp8(q, *cache, table, _i32(lens), window_left=left, o=o, lse=lse)
        assert torch.equal(a[0], o) and torch.equal(a[1], lse)


@pytest.mark.parametrize("new,left", [(1, -1), (1, 900), (6, -1), (512, -1), (512, 300)])
def test_table_as_wide_as_a_context(fl, new, left):
    """A table of 131072 keys over short sequences, anything in its unused entries: splits and parts by the table's
    width, most of them empty, and the same answers."""
    g = torch.Generator().manual_seed(29)
    page, hq, hkv, d, lens = 16, 8, 2, 128, [3000, 520, 37]
    width, pages = 131072 // page, sum(-(-x // page) for x in lens) + 2
    adds = [min(new, x) for x in lens]
    table = _table(lens, page, 200, pages, g)
    wide = torch.randint(-2 ** 31, 2 ** 31, (len(lens), width), generator=g, dtype=torch.int64).int()
    for b, n in enumerate(lens):
        held = -(-n // page)
        wide[b, :held] = torch.tensor(table[b][:held])
    cache = _cache(pages, page, hkv, d, g)
    q = torch.randn(sum(adds), hq, d, generator=g).to(torch.bfloat16)
    cu = [0] + torch.tensor(adds).cumsum(0).tolist()
    dev = [t.cuda() for t in cache]
    if new == 1:
        o, lse = fl.attn_decode_paged_fp8(q[:, :, None].cuda(), *dev, wide.cuda(), _i32(lens), window_left=left)
        o = o[:, :, 0]
    else:
        o, lse = fl.attn_fwd_paged_fp8(q.cuda(), *dev, wide.cuda(), _i32(lens), _i32(cu), max(adds), causal=True, window_left=left)
        lse = lse.T
    for b, n in enumerate(lens):
        k, v = [ref.gather(ref.value(cache[i]), cache[2 + i].double(), table[b], n) for i in range(2)]
        for i in sorted({0, adds[b] // 2, adds[b] - 1}):
            seen = n - adds[b] + i + 1
            exp = ref.attention(q[cu[b] + i][None].double(), k[:seen], v[:seen], float(torch.tensor(d ** -0.5, dtype=torch.float32)), left=left)
            _check_rows(o[cu[b] + i][None], lse[cu[b] + i][None], exp, d, seen, f"sequence {b}, token {i}")


# ---------------------------------------------------------------- as they are used
def _serve(fl, steps, page, hq, hkv, d, seed):
    """A prompt batch, then decode steps, then drafted tokens: every step plans, appends and attends."""
    g = torch.Generator().manual_seed(seed)
    B, width, pages = 3, 24, 60
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=g).int().cuda()
    cache = [torch.full((pages, page, hkv, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.full((pages, hkv), math.nan, device="cuda") for _ in range(2)]
    values = [torch.zeros(pages, page, hkv, d, dtype=torch.float64) for _ in range(2)]
    scales = [torch.zeros(pages, hkv, dtype=torch.float64) for _ in range(2)]
    host_lens, host_table, host_free = [0] * B, [[-1] * width for _ in range(B)], free.tolist()
    for new in steps:
        T = sum(new)
        slots, cu, out, counts = fl.attn_paged_plan(lens, _i32(new), free, table, page, T + 2)
        e = ref.plan(host_lens, new, host_free, host_table, page, T + 2)
        assert slots.tolist() == e[0] and table.tolist() == e[4] and counts.tolist() == e[3]
        kv = (torch.randn(T + 2, 2, hkv, d, generator=g) * torch.exp(torch.randn(T + 2, 1, 1, 1, generator=g))).to(torch.bfloat16)
        dkv = kv.cuda()
        fl.attn_append_paged_fp8(dkv[:, 0], dkv[:, 1], slots, *cache)
        for i in range(2):
            ref.append(kv[:, i].double(), e[0], values[i], scales[i])
        q = torch.randn(T, hq, d, generator=g).to(torch.bfloat16)
        if all(n == 1 for n in new):
            o, lse = fl.attn_decode_paged_fp8(q[:, :, None].cuda(), *cache, table, out)
            o = o[:, :, 0]
        else:
            o, lse = fl.attn_fwd_paged_fp8(q.cuda(), *cache, table, out, cu, max(new), causal=True)
            lse = lse.T
        lens, free = out, free[counts.tolist()[1]:].contiguous()
        host_lens, host_table, host_free = e[2], e[4], host_free[e[3][1]:]
        for b, n in enumerate(new):
            if n == 0:
                continue
            exp = ref.attention(q[e[1][b]:e[1][b + 1]].double(), ref.gather(values[0], scales[0], host_table[b], host_lens[b]),
                                ref.gather(values[1], scales[1], host_table[b], host_lens[b]), float(torch.tensor(d ** -0.5, dtype=torch.float32)))
            _check_rows(o[e[1][b]:e[1][b + 1]], lse[e[1][b]:e[1][b + 1]], exp, d, host_lens[b], f"step {new}, sequence {b}")


def test_serving_run(fl):
    _serve(fl, [[37, 5, 150], [1, 1, 1], [1, 1, 1], [4, 2, 3], [1, 1, 1], [60, 0, 17], [1, 1, 1]], 16, 8, 2, 128, seed=31)
    _serve(fl, [[200, 1, 90], [1, 1, 1], [130, 3, 0]], 64, 4, 4, 64, seed=32)


def test_without_native_calls(fl, monkeypatch):
    """The interpreted path of the four calls: the same bits."""
    g = torch.Generator().manual_seed(43)
    pages, page, hq, hkv, d = 20, 16, 8, 2, 128
    start = [t.cuda() for t in _cache(pages, page, hkv, d, g)]
    kv = torch.randn(70, 2, hkv, d, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(70, hq, d, generator=g).to(torch.bfloat16).cuda()

    def run():
        cache, table = [t.clone() for t in start], _i32([[0, 1] + [-1] * 6, [2] + [-1] * 7])
        plan = fl.attn_paged_plan(_i32([31, 16]), _i32([66, 4]), _i32(list(range(3, 20))), table, page, 70)
        fl.attn_append_paged_fp8(kv[:, 0], kv[:, 1], plan[0], *cache)
        return [*plan, table, *cache, *fl.attn_decode_paged_fp8(q[:2, :, None], *cache, table, plan[2]),
                *fl.attn_fwd_paged_fp8(q, *cache, table, plan[2], plan[1], 66, causal=True, window_left=50)]

    native = run()
    assert fl._calls is not None
    monkeypatch.setattr(fl, "_calls", None)
    for a, b in zip(native, run()):
        assert torch.equal(a, b)


def test_captured_step(fl):
    """Plan, append and decode in one CUDA graph: replays take the lengths and rows that the buffers hold then."""
    g = torch.Generator().manual_seed(41)
    B, page, hq, hkv, d, width, pages = 2, 16, 8, 2, 128, 8, 20
    table = _i32([[0, 1] + [-1] * 6, [2] + [-1] * 7])
    lens, new, free = _i32([31, 16]), _i32([1, 1]), _i32(list(range(3, 20)))
    cache = [t.cuda() for t in _cache(pages, page, hkv, d, g)]
    kv = torch.randn(B, 2, hkv, d, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(B, hq, 1, d, generator=g).to(torch.bfloat16).cuda()
    step = lambda: fl.attn_paged_plan(lens, new, free, table, page, B)  # noqa: E731

    def run():
        slots, cu, out, counts = step()
        fl.attn_append_paged_fp8(kv[:, 0], kv[:, 1], slots, *cache)
        return fl.attn_decode_paged_fp8(q, *cache, table, out) + (out, counts)

    start = [t.clone() for t in [table, lens, free, *cache]]

    def reset():
        for t, s in zip([table, lens, free, *cache], start):
            t.copy_(s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    inputs = [(torch.randn_like(kv), torch.randn_like(q)) for _ in range(3)]
    seen = []
    for x, y in inputs:
        kv.copy_(x), q.copy_(y)
        graph.replay()
        seen.append([t.clone() for t in held])
        lens.copy_(held[2])
        n = int(held[3][1])
        free[:free.numel() - n] = free[n:].clone()
    reset()
    for (x, y), got in zip(inputs, seen):
        kv.copy_(x), q.copy_(y)
        want = run()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        lens.copy_(want[2])
        n = int(want[3][1])
        free[:free.numel() - n] = free[n:].clone()


def test_captured_parts(fl):
    """Splits and parts that merge through memory, captured; two graphs that share the workspaces, replayed in turn over
    new lengths and queries."""
    g = torch.Generator().manual_seed(44)
    page, hq, hkv, d, width = 16, 8, 2, 128, 400
    table = _i32([torch.randperm(500, generator=g)[:width].tolist()])
    cache = [t.cuda() for t in _cache(500, page, hkv, d, g)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def made(new):
        st = dict(q=torch.randn(new, hq, d, generator=g).to(torch.bfloat16).cuda(), lens=_i32([6000]), cu=_i32([0, new]))
        st["o"], st["lse"] = torch.empty_like(st["q"]), torch.empty(hq, new, device="cuda")
        st["do"], st["dlse"] = torch.empty(1, hq, 1, d, dtype=torch.bfloat16, device="cuda"), torch.empty(1, hq, device="cuda")
        return st

    def run(st, **kw):
        a = fl.attn_fwd_paged_fp8(st["q"], *cache, table, st["lens"], st["cu"], len(st["q"]), causal=True, **kw)
        kw.update({k: st["d" + k] for k in ("o", "lse") if k in kw})
        return [*a, *fl.attn_decode_paged_fp8(st["q"][:1, :, None], *cache, table, st["lens"], num_splits=12, **kw)]

    states = [made(70), made(5)]
    graphs = []
    for st in states:
        run(st)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run(st, o=st["o"], lse=st["lse"], workspace=ws)
    for step in range(6):
        st = states[step % 2]
        st["lens"].fill_(6400 - 900 * step)
        st["q"].copy_(torch.randn(st["q"].shape, generator=g))
        graphs[step % 2].replay()
        for a, b in zip((st["o"], st["lse"], st["do"], st["dlse"]), run(st)):
            assert torch.equal(a, b), step


def test_host_threads(fl):
    """Calls from several host threads, each on a stream of its own."""
    g = torch.Generator().manual_seed(45)
    lens, page = [3000, 2500], 16
    pages = sum(-(-x // page) for x in lens)
    table, held = _i32(_table(lens, page, 190, pages, g)), _i32(lens)
    cache = [t.cuda() for t in _cache(pages, page, 2, 128, g)]
    qs = [torch.randn(120, 8, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(4)]
    cu = _i32([0, 60, 120])
    want = [fl.attn_fwd_paged_fp8(q, *cache, table, held, cu, 60, causal=True) for q in qs]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for turn in range(10):
                got[i] = fl.attn_fwd_paged_fp8(qs[i], *cache, table, held, cu, 60, causal=True,
                                               workspace=None if turn % 2 else torch.empty(8 << 20, dtype=torch.uint8, device="cuda"))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_other_stream(fl):
    """Calls on a side stream, two at once with workspaces of their own."""
    g = torch.Generator().manual_seed(42)
    lens, page = [3000, 2500], 16
    pages = sum(-(-x // page) for x in lens)
    table = _i32(_table(lens, page, 190, pages, g))
    cache = [t.cuda() for t in _cache(pages, page, 2, 128, g)]
    qs = [torch.randn(2, 8, 1, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [fl.attn_decode_paged_fp8(q, *cache, table, _i32(lens)) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        got = []
        for s, q in zip(streams, qs):
            with torch.cuda.stream(s):
                got.append(fl.attn_decode_paged_fp8(q, *cache, table, _i32(lens)))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
