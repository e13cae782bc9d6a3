"""The attention operators against their plain 64-bit forms (tests/attn_ref.py
derives the attention tolerances)."""
import math

import pytest
import torch

import attn_ref as R
import bit_dequant_expert_b200 as m

pytestmark = pytest.mark.gpu


def rng(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ prepare


def prepare_case(T, hq, hkv, dim, rot, layout, e4m3, page, seed, scale=1.0, norm=True, first=0, extra=0, skip=False):
    g = rng(seed)
    qkv = (torch.randn(T, (hq + 2 * hkv) * dim + extra, generator=g) * 3).bfloat16()
    qw, kw = ((1 + 0.2 * torch.randn(dim, generator=g)).bfloat16() for _ in range(2))
    if not norm:
        qw = kw = None
    inv = torch.pow(10000.0, -torch.arange(0, rot, 2).double() / max(rot, 1)).float() if rot else None
    pos = (torch.arange(T) * 3 + first).int()
    pages = (T + page - 1) // page + 1
    slots = torch.randperm(pages * page, generator=g)[:T].int()
    if skip:
        slots[::3] = -1
    return dict(qkv=qkv, qw=qw, kw=kw, inv=inv, pos=pos, slots=slots, pages=pages, rs=scale)


def run_prepare(c, d, T, rot, layout, k_out=True, slots=True, err=None, stride=None):
    hq, hkv, dim, page = c.q_heads, c.kv_heads, c.head_dim, c.page_size
    e4m3 = c.cache_type == m.ATTN_CACHE_E4M3
    shape = (d["pages"], hkv, page, dim)
    fill = 7.0   # what is not written stays
    kc, vc = (torch.full(shape, fill, device="cuda").to(torch.float8_e4m3fn if e4m3 else torch.bfloat16) for _ in "kv")
    ks, vs = (torch.full(shape[:3], fill, device="cuda") if e4m3 else None for _ in "kv")
    q = torch.full((T, hq, dim), math.nan, dtype=torch.bfloat16, device="cuda")
    k = torch.full((T, hkv, dim), math.nan, dtype=torch.bfloat16, device="cuda") if k_out else None
    qkv, qw, kw, inv, pos, sl = R.cuda(d["qkv"], d["qw"], d["kw"], d["inv"], d["pos"], d["slots"])
    m.attn_qkv_prepare(c, T, qkv, qkv.stride(0), qw, kw, 1e-6, inv, rot, layout, d["rs"], pos, sl if slots else None,
                       d["pages"], kc, vc, ks, vs, q, k, err=err)
    torch.cuda.synchronize()
    return q, k, kc, vc, ks, vs


def check_prepared(c, d, T, rot, layout, got):
    hq, hkv, dim, page = c.q_heads, c.kv_heads, c.head_dim, c.page_size
    (q, qs), (k, ksz), v = R.prepared(d["qkv"][:, :(hq + 2 * hkv) * dim], hq, hkv, dim, d["qw"], d["kw"], 1e-6,
                                      d["inv"], rot, layout, d["rs"], d["pos"])
    gq, gk, kc, vc, ks, vs = [None if t is None else t.cpu() for t in got]
    # fp32 arithmetic: the sum of squares of up to 256 terms, the root and its product, the angle and two products:
    # under 2^-18 of the sizes; then one rounding, half a step
    def close(x, ref, size):
        off = (x.double() - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -18 * size)
        assert off.max() <= 0, "off by %.3e more than allowed" % off.max()

    close(gq, q, qs)
    if gk is not None:
        close(gk, k, ksz)
    slots = d["slots"].long()
    live = slots >= 0
    p, o = slots[live] // page, slots[live] % page
    touched = torch.zeros(d["pages"], page, dtype=torch.bool)
    touched[p, o] = True
    for cache, scale, ref, size in ((kc, ks, k, ksz), (vc, vs, v, v.abs())):
        rows = cache.float()[p, :, o].double()
        ref, size = ref[live], size[live]
        if scale is None:
            off = (rows - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -18 * size)
        else:
            s = scale[p, :, o].double()
            want = ref.abs().amax(-1) / 448
            want = torch.where(want > 0, want, torch.ones_like(want))
            assert ((s - want).abs() <= 2.0 ** -18 * want + 2.0 ** -18 * size.amax(-1) / 448).all()
            # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale among the subnormals
            half = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * s[..., None])
            off = (rows * s[..., None] - ref).abs() - half * (1 + 2.0 ** -16) - 2.0 ** -17 * size
        assert off.numel() == 0 or off.max() <= 0, "cache off by %.3e more than allowed" % off.max()
        assert (cache.float().transpose(1, 2)[~touched] == 7.0).all(), "rows outside the slots changed"


@pytest.mark.parametrize("T,hq,hkv,dim,rot,layout,e4m3,page,kw", [
    (1, 16, 2, 128, 128, 0, True, 64, {}),
    (1, 16, 2, 256, 64, 0, False, 16, dict(first=1_000_003)),
    (7, 5, 1, 64, 64, 1, True, 16, dict(norm=False)),
    (33, 12, 4, 128, 48, 1, False, 128, dict(scale=1.2, extra=24)),
    (300, 8, 8, 64, 16, 0, True, 32, dict(skip=True)),
    (65, 16, 2, 256, 256, 0, True, 16, dict(first=2_000_000_000, scale=0.7)),
    (50, 3, 3, 128, 0, 0, True, 64, {}),
    (2500, 16, 2, 128, 128, 1, True, 64, dict(first=65536)),
    (1300, 32, 8, 64, 32, 0, False, 32, dict(skip=True)),
    (40, 16, 2, 128, 96, 1, True, 16, dict(first=-70)),      # positions below zero too
])
def test_prepare(T, hq, hkv, dim, rot, layout, e4m3, page, kw):
    c = m.attn_config(hq, hkv, dim, page, int(e4m3))
    d = prepare_case(T, hq, hkv, dim, rot, layout, e4m3, page, T + dim, **kw)
    got = run_prepare(c, d, T, rot, layout)
    check_prepared(c, d, T, rot, layout, got)
    # without the keys' copy, and without a cache: the same outputs
    q, k, *_ = run_prepare(c, d, T, rot, layout, k_out=False)
    assert k is None and torch.equal(q, got[0])
    q, k, kc, *_ = run_prepare(c, d, T, rot, layout, slots=False)
    assert torch.equal(q, got[0]) and torch.equal(k, got[1]) and (kc.float() == 7.0).all()


def test_prepare_edge_rows_and_bad_slots():
    """A row of zeros (scale 1, codes 0), rows with an infinity or NaN (scale
    NaN), tiny and huge rows, and slots past the cache (reported, skipped)."""
    c = m.attn_config(4, 2, 128, 16, m.ATTN_CACHE_E4M3)
    d = prepare_case(8, 4, 2, 128, 0, 0, True, 16, 3, norm=False)
    rows = d["qkv"].view(8, 8, 128)
    rows[0, 4:] = 0
    rows[1, 4:, 5] = math.inf
    rows[2, 6:, 7] = math.nan
    rows[3, 4:] *= 1e-38
    rows[4, 4:] *= 1e37
    d["slots"] = torch.tensor([0, 1, 2, 3, 4, 5, d["pages"] * 16, 2 ** 31 - 1], dtype=torch.int32)
    err = err_word()
    q, k, kc, vc, ks, vs = run_prepare(c, d, 8, 0, 0, err=err)
    assert err.item() == m.MOE_ERR_BOUNDS
    assert torch.equal(q.cpu(), rows[:, :4])
    assert (ks[0, :, 0] == 1).all() and (vs[0, :, 0] == 1).all() and (kc.float()[0, :, 0] == 0).all()
    assert ks[0, :, 1].isnan().all() and vs[0, :, 1].isnan().all()
    assert vs[0, :, 2].isnan().all() and not ks[0, :, 2].isnan().any()
    for t in (3, 4, 5):
        ref = rows[t, 4:6].double()
        got = (kc.float()[0, :, t].double() * ks[0, :, t, None].double()).cpu()
        assert ((got - ref).abs() <= 2.0 ** -4 * ref.abs() * 1.0001 + ks[0, :, t, None].cpu().double() * 2.0 ** -10 + 1.5e-45 * 448).all()
    assert (kc.float()[0, :, 6:] == 7.0).all()


# ------------------------------------------------------------------ read


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prepare_codes_are_those_of_a_division(dim):
    """Value rows of every size, ties among them: code for code what a 32-bit
    division and one rounding to nearest even give."""
    g, T, hkv, page = rng(dim), 4096, 2, 64
    v = torch.randn(T, hkv, dim, generator=g)
    v[::3] = torch.randint(-448, 449, v[::3].shape, generator=g).float() / 32   # quotients on and next to borders
    v *= torch.exp2(torch.randint(-126, 121, (T, hkv, 1), generator=g).float())
    v[5], v[7, :, 1:] = 0.0, 0.0
    v = v.bfloat16()
    qkv = torch.cat([torch.zeros(T, (1 + hkv) * hkv * dim, dtype=torch.bfloat16), v.flatten(1)], 1).cuda()
    c = m.attn_config(hkv * hkv, hkv, dim, page, m.ATTN_CACHE_E4M3)
    kc, vc = (torch.zeros(T // page, hkv, page, dim, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(T // page, hkv, page, device="cuda") for _ in range(2))
    q = torch.empty(T, hkv * hkv, dim, dtype=torch.bfloat16, device="cuda")
    m.attn_qkv_prepare(c, T, qkv, qkv.stride(0), None, None, 0.0, None, 0, 0, 1.0, None,
                       torch.arange(T, dtype=torch.int32, device="cuda"), T // page, kc, vc, ks, vs, q, None)
    torch.cuda.synchronize()
    codes, scales = (t.cpu().transpose(1, 2).flatten(0, 1) for t in (vc.view(torch.uint8), vs))
    want, s = R.quantised(v.float())
    normal = (s >= 2.0 ** -126) & torch.isfinite(s)      # scales that are numbers of full precision
    assert normal.float().mean() > 0.9 and torch.equal(scales[normal], s[normal])
    assert torch.equal(codes[normal], want.view(torch.uint8)[normal])


@pytest.mark.parametrize("lens,hkv,dim,e4m3,page", [
    ([1], 2, 128, True, 64), ([0, 33, 0, 1, 128, 0], 1, 64, True, 16), ([257, 64, 63], 8, 256, False, 32),
    ([777], 2, 256, True, 128), ([5, 700, 31, 1], 3, 128, False, 64), (list(range(0, 40)), 2, 64, False, 16)])
def test_read(lens, hkv, dim, e4m3, page):
    g = rng(sum(lens))
    table, pages = R.make_table(g, lens, page)
    kc, vc, ks, vs = R.make_cache(g, pages, hkv, page, dim, e4m3)
    total = sum(lens)
    cu = R.starts(lens) + 2      # two rows before the first sequence and three after the last stay
    c = m.attn_config(hkv, hkv, dim, page, int(e4m3))
    k = torch.full((total + 5, hkv, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    tb, cu_d, kd, vd, ksd, vsd = R.cuda(table, cu, kc, vc, ks, vs)
    err = err_word()
    m.attn_kv_read(c, len(lens), total + 5, tb, tb.stride(0), cu_d, pages, kd, vd, ksd, vsd, k, v, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for got, cache, scale in ((k, kc, ks), (v, vc, vs)):
        ref = torch.cat([R.rows_of(cache, scale, table[b], n) for b, n in enumerate(lens)])
        got = got.cpu()
        assert (got[:2] == 9.0).all() and (got[total + 2:] == 9.0).all()
        # the product code * scale has one fp32 rounding (2^-24) before the one to bf16
        assert ((got[2:total + 2].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all()


def test_read_reports_bad_pages_and_lengths():
    g = rng(1)
    table, pages = R.make_table(g, [40, 40], 16)
    kc, vc, _, _ = R.make_cache(g, pages, 2, 16, 64, False)
    c = m.attn_config(2, 2, 64, 16, 0)
    table[0, 1], table[1, 0] = pages, -1
    tb, kd, vd = R.cuda(table, kc, vc)

    def call(cu, total):
        err = err_word()
        k = torch.full((total, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        v = k.clone()
        m.attn_kv_read(c, 2, total, tb, 3, torch.tensor(cu, dtype=torch.int32).cuda(), pages, kd, vd, None, None, k, v,
                       err=err)
        torch.cuda.synchronize()
        return err.item(), k.cpu()

    status, k = call([0, 40, 80], 80)
    assert status == m.MOE_ERR_BOUNDS and (k[16:32] == 0).all() and (k[40:56] == 0).all()
    assert torch.equal(k[:16], kc[table[0, 0].long()].transpose(0, 1))
    table[0, 1], table[1, 0] = 0, 1
    tb.copy_(table)
    assert call([0, 40, 80], 80)[0] == 0
    assert call([0, 40, 80], 70)[0] == m.MOE_ERR_BOUNDS       # more rows than the outputs hold
    status, k = call([0, 49, 80], 80)                         # longer than its row of pages
    assert status == m.MOE_ERR_BOUNDS and (k[48] == 0).all()


# ------------------------------------------------------------------ prefill


def prefill_limit(nq, nk, causal):
    return [max(0, min(nk, nk - nq + i + 1)) if causal else nk for i in range(nq)]


def run_prefill(lens_q, lens_k, hq, hkv, dim, causal, seed, gain=1.5, pad=0, scale=None, data=None):
    g = rng(seed)
    tq, tk = sum(lens_q), sum(lens_k)
    q = (torch.randn(tq + 3, hq, dim, generator=g) * gain).bfloat16()
    k = (torch.randn(tk + 2, hkv, dim, generator=g) * gain).bfloat16()
    v = torch.randn(tk + 2, hkv, dim, generator=g).bfloat16()
    if data:
        data(q, k, v)
    scale = dim ** -0.5 if scale is None else scale
    cu_q, cu_k = R.starts(lens_q) + 1, R.starts(lens_k) + 2   # rows before and behind belong to nobody
    c = m.attn_config(hq, hkv, dim)
    wide = lambda t, w: torch.cat([t.flatten(1), torch.full((t.shape[0], w), math.nan).bfloat16()], 1).cuda()  # noqa: E731
    qd, kd, vd = wide(q, pad), wide(k, 2 * pad), wide(v, pad)
    out = torch.full((tq + 3, hq, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((tq + 3, hq), 5.0, device="cuda")
    err = err_word()
    m.attn_prefill(c, len(lens_q), tq + 3, tk + 2, cu_q.cuda(), cu_k.cuda(), qd, qd.stride(0), kd, kd.stride(0), vd,
                   vd.stride(0), scale, causal, out, lse, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for t in (out, lse):
        assert (t[:1] == 5.0).all() and (t[tq + 1:] == 5.0).all(), "rows of no sequence changed"
    for b in range(len(lens_q)):
        r, s = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        if lens_q[b]:
            ref = R.attend(q[r], k[s], v[s], scale, prefill_limit(lens_q[b], lens_k[b], causal))
            R.check_attention(out[r].cpu(), lse[r].cpu(), ref)
    return out, lse


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens_q,lens_k,hq,hkv", [
    ([1], [1], 2, 1),
    ([127], [127], 2, 2),
    ([128], [128], 4, 1),
    ([129], [129], 1, 1),
    ([300], [300], 16, 2),
    ([1, 64, 0, 200, 3], [1, 64, 0, 200, 3], 4, 2),
    ([5, 130, 17], [400, 131, 257], 3, 1),            # chunks after a prefix; three heads of one key head
    ([200, 40, 7], [60, 0, 3], 2, 1),                 # fewer keys than queries, and none at all
    ([513], [1030], 5, 1),
    ([255, 256, 257], [255, 256, 257], 6, 2),
])
def test_prefill(lens_q, lens_k, hq, hkv, dim, causal):
    run_prefill(lens_q, lens_k, hq, hkv, dim, causal, seed=sum(lens_q) + dim)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prefill_strides_and_scales(dim):
    run_prefill([70, 130], [70, 200], 4, 2, dim, True, 5, pad=40)
    run_prefill([70, 130], [70, 200], 4, 2, dim, True, 6, gain=6.0)              # one key takes nearly all
    run_prefill([150], [300], 2, 2, dim, False, 7, scale=-0.1)
    run_prefill([150], [300], 2, 2, dim, False, 7, scale=0.0)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prefill_rising_scores(dim):
    """Scores that grow along the keys by hundreds, so that the running maximum
    moves in every tile; and keys far below the rest."""
    def rising(q, k, v):
        q[:] = 0
        q[..., 0] = 8
        k[..., 0] = torch.arange(k.shape[0])[:, None] * 0.5

    run_prefill([200], [600], 2, 1, dim, False, 8, scale=0.25, data=rising)
    run_prefill([600], [600], 2, 1, dim, True, 9, scale=0.25, data=rising)
    run_prefill([600], [600], 2, 1, dim, True, 10, scale=-0.25, data=rising)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prefill_neighbours_do_not_leak(dim):
    """Rows of no sequence and of other sequences that hold NaN and infinities
    change nothing."""
    lens = [100, 60, 200]

    def poison(q, k, v):
        for t in (k, v):
            t[0], t[1] = math.nan, math.inf
            t[102:162] = math.nan          # the middle sequence's rows
            t[362:] = math.nan             # behind the last sequence

    g = rng(11)
    q = torch.randn(363, 4, dim, generator=g).bfloat16()
    k, v = (torch.randn(365, 2, dim, generator=g).bfloat16() for _ in "kv")
    clean = [t.clone() for t in (k, v)]
    poison(q, k, v)
    c = m.attn_config(4, 2, dim)
    cu_q, cu_k = (R.starts(lens) + 1).cuda(), (R.starts(lens) + 2).cuda()
    outs = []
    for kk, vv in (clean, (k, v)):
        qd, kd, vd = R.cuda(q, kk, vv)
        out = torch.zeros(363, 4, dim, dtype=torch.bfloat16, device="cuda")
        m.attn_prefill(c, 3, 363, 365, cu_q, cu_k, qd, 4 * dim, kd, 2 * dim, vd, 2 * dim, 0.1, True, out)
        torch.cuda.synchronize()
        outs.append(out.cpu())
    assert torch.equal(outs[0][:101], outs[1][:101]) and torch.equal(outs[0][161:], outs[1][161:])
    assert outs[1][101:161].isnan().all()


def cold_prefills(lens_q, lens_k, hq, hkv, dim, causal, seed, repeats=6, data=None, scale=None):
    """The same call again and again, each time after 256 MB were read, so that
    its loads arrive at uneven times: each gives the same bits, and what the
    definition says."""
    g = rng(seed)
    q = (torch.randn(sum(lens_q), hq, dim, generator=g) * 1.5).bfloat16()
    k = (torch.randn(sum(lens_k), hkv, dim, generator=g) * 1.5).bfloat16()
    v = torch.randn(sum(lens_k), hkv, dim, generator=g).bfloat16()
    if data:
        data(q, k)
    scale = dim ** -0.5 if scale is None else scale
    c, cu_q, cu_k = m.attn_config(hq, hkv, dim), R.starts(lens_q), R.starts(lens_k)
    qd, kd, vd, cq, ck = R.cuda(q, k, v, cu_q, cu_k)
    err, cold, first = err_word(), torch.zeros(64 << 20, device="cuda"), None
    for _ in range(repeats):
        cold.sum()                                       # more than the cache holds
        out = torch.full(q.shape, math.nan, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:2], math.nan, device="cuda")
        m.attn_prefill(c, len(lens_q), q.shape[0], k.shape[0], cq, ck, qd, hq * dim, kd, hkv * dim, vd, hkv * dim, scale,
                       causal, out, lse, err=err)
        torch.cuda.synchronize()
        assert err.item() == 0
        if first is None:
            first = (out, lse)
            for b in range(len(lens_q)):
                r, s = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
                if lens_q[b]:
                    ref = R.attend(q[r], k[s], v[s], scale, prefill_limit(lens_q[b], lens_k[b], causal))
                    R.check_attention(out[r].cpu(), lse[r].cpu(), ref)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens_q,lens_k,hq,hkv", [
    ([256], [256], 48, 48),                              # two blocks of keys
    ([140, 5], [200, 5], 256, 256),
    ([1, 128, 129, 300, 400, 640, 700], [1, 128, 129, 300, 400, 640, 700], 24, 24),   # one to six blocks
    ([130, 257], [700, 511], 64, 8),                     # chunks after a prefix
    ([300], [300], 8, 2),                                # few tiles
    ([640], [760], 4, 4),
])
def test_prefill_from_cold_memory(lens_q, lens_k, hq, hkv, dim, causal):
    cold_prefills(lens_q, lens_k, hq, hkv, dim, causal, seed=sum(lens_k) + dim)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("high", range(1, 6))
def test_prefill_maximum_moves_before_the_last_block(dim, high):
    """Scores are 0 but in one block of keys, where they are some 30 above: of
    the row's maxima only that block's moves, and every later block, the last
    one too, works with the maximum that it was handed."""
    def raised(q, k):
        q[:], k[:] = 0, 0
        q[..., 0] = 4
        k[high * 128 - 100:high * 128, :, 0] = (8 + torch.arange(100)[:, None] / 128).bfloat16()

    blocks = high + 1
    cold_prefills([128], [blocks * 128 - 3], 148, 148, dim, False, high, data=raised, scale=1.0)
    cold_prefills([200, 128], [700, blocks * 128], 64, 8, dim, False, high, data=raised, scale=1.0)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prefill_calls_in_a_row(dim):
    """Hundreds of short blocks after one another on each multiprocessor, call
    upon call: the same bits in every one."""
    hq, hkv, lens = 48, 24, [130, 17, 128, 260, 1, 64] * 8
    g = rng(dim)
    cu = R.starts(lens).cuda()
    q, k, v = ((torch.randn(sum(lens), h, dim, generator=g)).bfloat16().cuda() for h in (hq, hkv, hkv))
    c, err = m.attn_config(hq, hkv, dim), err_word()
    outs = [torch.full(q.shape, math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(12)]
    for out in outs:
        m.attn_prefill(c, len(lens), q.shape[0], q.shape[0], cu, cu, q, hq * dim, k, hkv * dim, v, hkv * dim, dim ** -0.5,
                       True, out, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.isfinite(outs[0].float()).all()
    assert all(torch.equal(out, outs[0]) for out in outs[1:])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,seqs", [(64, 64, 4), (48, 16, 4), (64, 32, 4), (3, 1, 1), (2, 2, 1)])
@pytest.mark.parametrize("lq,lk", [(256, 320), (150, 214), (400, 401), (257, 384), (300, 300)])
def test_prefill_non_finite_values_reach_back_127_positions(lq, lk, hq, hkv, seqs, dim):
    """One value row of a head holds NaN: queries that see it give NaN, those
    more than 127 positions before it what the definition says of the rows that
    they see, wherever the row lies in a tile."""
    g, c = rng(lk + hq), m.attn_config(hq, hkv, dim)
    q = torch.randn(seqs * lq, hq, dim, generator=g).bfloat16()
    k, v = (torch.randn(seqs * lk, hkv, dim, generator=g).bfloat16() for _ in "kv")
    scale, cu_q, cu_k = dim ** -0.5, R.starts([lq] * seqs).cuda(), R.starts([lk] * seqs).cuda()
    qd, kd = R.cuda(q, k)
    for at in sorted({lk - 1, lk - lq + 128, lk - lq + 191, 255, 128, min(lk - 1, 300)}):
        if at >= seqs * lk:
            continue
        bad = v.clone()
        bad[at] = math.nan
        out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
        m.attn_prefill(c, seqs, seqs * lq, seqs * lk, cu_q, cu_k, qd, hq * dim, kd, hkv * dim, bad.cuda(), hkv * dim, scale,
                       True, out)
        got, b = out.cpu().split(lq), at // lk
        first = at - b * lk - (lk - lq)                      # the first query of sequence b that sees the row
        before = max(0, min(lq, first - 127))
        if before:
            r = slice(b * lq, b * lq + before)
            ref = R.attend(q[r], k[b * lk:(b + 1) * lk], v[b * lk:(b + 1) * lk], scale, prefill_limit(lq, lk, True)[:before])
            R.check_attention(got[b][:before], None, ref)
        assert got[b][max(0, first):].isnan().all()
        assert all(o.isfinite().all() for i, o in enumerate(got) if i != b)


def test_prefill_reports_bad_boundaries():
    c = m.attn_config(2, 1, 64)
    q, k = torch.ones(20, 2, 64, device="cuda").bfloat16(), torch.ones(20, 1, 64, device="cuda").bfloat16()
    for cu_q, cu_k in (([0, 10, 20], [0, 10, 21]), ([0, 10, 20], [0, 10, 5]), ([0, 10, 21], [0, 10, 20]),
                       ([0, 10, 20], [-1, 0, 20]), ([-5, 10, 20], [0, 10, 20]), ([0, 10, 4], [0, 10, 20])):
        out = torch.full((20, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        err = err_word()
        m.attn_prefill(c, 2, 20, 20, *(torch.tensor(t, dtype=torch.int32).cuda() for t in (cu_q, cu_k)), q, 128, k, 64,
                       k, 64, 0.1, False, out, err=err)
        torch.cuda.synchronize()
        assert err.item() == m.MOE_ERR_BOUNDS
        bad_first = cu_q[0] < 0 or cu_k[0] < 0
        assert (out[:10] == (5.0 if bad_first else 1.0)).all()
        if not bad_first:
            assert (out[10:] == 5.0).all()


def test_prefill_many_sequences():
    """More sequences than a block has threads, most of one token."""
    g = rng(12)
    lens = [int(n) for n in torch.randint(0, 4, (1500,), generator=g)]
    run_prefill(lens, lens, 2, 1, 64, True, 13)


# ------------------------------------------------------------------ decode


def run_decode(lens, nq, hq, hkv, dim, e4m3, page, seed, max_len=None, gain=1.5, poison=True, ws_extra=0):
    g = rng(seed)
    table, pages = R.make_table(g, lens, page)
    kc, vc, ks, vs = R.make_cache(g, pages, hkv, page, dim, e4m3)
    q = (torch.randn(len(lens) * nq, hq, dim, generator=g) * gain).bfloat16()
    scale = dim ** -0.5
    kd, vd, ksd, vsd = R.cuda(kc, vc, ks, vs)
    if poison:   # rows past each sequence's end, and pages of no sequence
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            j = torch.arange(n)
            used[table[b].long()[j // page], j % page] = True
        free = (~used)[:, None, :].expand(pages, hkv, page).cuda()
        for t in (kd, vd):
            if e4m3:
                t.view(torch.uint8)[free] = 0x7F      # NaN
            else:
                t[free] = math.nan
        for t in (ksd, vsd):
            if t is not None:
                t[free] = math.nan
    c = m.attn_config(hq, hkv, dim, page, int(e4m3))
    top = max(lens + [1]) if max_len is None else max_len
    need = (top + page - 1) // page
    if table.shape[1] < need:
        table = torch.cat([table, torch.full((len(lens), need - table.shape[1]), -7, dtype=torch.int32)], 1)
    ws = torch.full((m.attn_decode_workspace_size(c, len(lens), nq, top) + ws_extra,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((len(lens) * nq, hq, dim), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((len(lens) * nq, hq), math.nan, device="cuda")
    err = err_word()
    qd, tb, ln = R.cuda(q, table, torch.tensor(lens, dtype=torch.int32))
    m.attn_decode(c, len(lens), nq, top, qd, hq * dim, tb, tb.stride(0), ln, pages, kd, vd, ksd, vsd, scale, out, lse,
                  ws, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for b, n in enumerate(lens):
        r = slice(b * nq, b * nq + nq)
        ref = R.attend(q[r], R.rows_of(kc, ks, table[b], n), R.rows_of(vc, vs, table[b], n), scale,
                       [max(0, n - nq + i + 1) for i in range(nq)])
        R.check_attention(out[r].cpu(), lse[r].cpu(), ref)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,nq,hq,hkv,page", [
    ([1], 1, 1, 1, 16),
    ([63, 64, 65], 1, 16, 2, 64),
    ([0, 17, 1, 300], 1, 4, 4, 16),
    ([1000], 1, 16, 2, 128),
    ([5, 130, 1], 4, 16, 2, 32),          # verification rows; a sequence shorter than its new tokens
    ([257, 700], 8, 8, 1, 64),            # 64 query rows of one key head
    ([190], 3, 5, 1, 16),
    ([2049, 31], 2, 12, 4, 32),
    ([129], 8, 32, 2, 16),                # 128 query rows of one key head
])
def test_decode(lens, nq, hq, hkv, page, dim, e4m3):
    run_decode(lens, nq, hq, hkv, dim, e4m3, page, seed=sum(lens) + dim)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_long_and_loose_bounds(e4m3):
    run_decode([20000], 1, 16, 2, 128, e4m3, 64, 1)
    run_decode([7, 20001, 5000], 2, 4, 1, 256, e4m3, 16, 2)
    run_decode([7, 300], 1, 4, 2, 128, e4m3, 16, 3, max_len=100_000)      # max_len far above every length
    run_decode([500], 1, 16, 2, 128, e4m3, 64, 4, gain=8.0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_many_sequences(e4m3):
    """More sequences than a block has threads, short and empty ones among
    them, and one long one behind them."""
    g = rng(14)
    lens = [int(n) for n in torch.randint(0, 90, (450,), generator=g)] + [3000, 0, 1]
    run_decode(lens, 1, 2, 1, 64, e4m3, 16, 15)
    run_decode(lens[200:], 3, 16, 2, 128, e4m3, 32, 16)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("nq", [1, 2, 4, 8])
def test_decode_long_runs_from_cold_memory(nq, dim, e4m3):
    """Runs of many tiles whose loads arrive at uneven times (a cold cache,
    pages in any order, some of them shared): each call gives the same bits,
    and what the definition says."""
    hq, hkv, page, pages = 16, 2, 64, 1500
    g = torch.Generator(device="cuda").manual_seed(nq + dim)
    lens = [int(n) for n in torch.randint(1, 8193, (40,), generator=rng(nq))] + [100, 1500]
    kc, vc = (torch.randn(pages, hkv, page, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    ks = vs = None
    if e4m3:
        (kc, ks), (vc, vs) = R.quantised(kc.float()), R.quantised(vc.float())
    table = torch.randint(0, pages, (len(lens), 128), generator=g, device="cuda", dtype=torch.int32)
    q = (torch.randn(len(lens) * nq, hq, dim, generator=g, device="cuda") * 1.5).bfloat16()
    c, top = m.attn_config(hq, hkv, dim, page, int(e4m3)), max(lens)
    ws = torch.empty(m.attn_decode_workspace_size(c, len(lens), nq, top), dtype=torch.uint8, device="cuda")
    ln, err, cold = torch.tensor(lens, dtype=torch.int32, device="cuda"), err_word(), torch.zeros(64 << 20, device="cuda")
    first = None
    for _ in range(6):
        cold.sum()                                       # 256 MB: more than the cache holds
        out = torch.full((len(lens) * nq, hq, dim), math.nan, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((len(lens) * nq, hq), math.nan, device="cuda")
        assert m.attn_decode(c, len(lens), nq, top, q, hq * dim, table, table.stride(0), ln, pages, kc, vc, ks, vs,
                             dim ** -0.5, out, lse, ws, err=err) == 0
        torch.cuda.synchronize()
        assert err.item() == 0
        first = first or (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    for b in (len(lens) - 2, len(lens) - 1):
        used = table[b, :(lens[b] + page - 1) // page].long()
        rows = [R.rows_of(x[used].cpu(), None if s is None else s[used].cpu(), torch.arange(len(used)), lens[b])
                for x, s in ((kc, ks), (vc, vs))]
        r = slice(b * nq, b * nq + nq)
        ref = R.attend(q[r].cpu(), *rows, dim ** -0.5, [lens[b] - nq + i + 1 for i in range(nq)])
        R.check_attention(first[0][r].cpu(), first[1][r].cpu(), ref)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("nq,hq,hkv", [(8, 64, 1), (1, 256, 4), (3, 256, 256)])
def test_decode_most_heads(nq, hq, hkv, dim, e4m3):
    """The largest counts of heads and of query rows of one key head."""
    run_decode([70, 0, 300], nq, hq, hkv, dim, e4m3, 16, seed=hq + nq)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_cache_most_heads(dim, e4m3):
    for T, hq, hkv in ((1, 256, 256), (70, 256, 4), (5, 64, 64)):
        test_prepare(T, hq, hkv, dim, dim, T % 2, e4m3, 16, {})
        test_read([T, 0, 33], hkv, dim, e4m3, 16)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(64, 1), (256, 4), (256, 256)])
def test_prefill_most_heads(hq, hkv, dim):
    run_prefill([5, 0, 140], [5, 3, 200], hq, hkv, dim, True, seed=hq)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("nq", [1, 4])
def test_decode_small_values_beside_rows_of_zeros(nq, dim):
    """A row of zeros has the scale 1, the rows beside it 2.4 2^-24: their
    probabilities keep their bits (half a step of 2^-32 of the largest: 0.07%
    here, within the 2^-8 that check_attention allows a probability)."""
    g, page, lens, hkv = rng(nq), 64, [600, 77], 2
    table, pages = R.make_table(g, lens, page)
    kc, ks = R.quantised(torch.randn(pages, hkv, page, dim, generator=g))
    v = torch.randn(dim, generator=g)
    v = (v * (448 * 2.4 * 2.0 ** -24 / v.abs().max())).expand(pages, hkv, page, dim).clone()
    v[:, :, 1::2] = 0.0
    vc, vs = R.quantised(v)
    assert (vs[:, :, 1::2] == 1.0).all()
    q = torch.zeros(len(lens) * nq, 16, dim, dtype=torch.bfloat16)    # every key counts alike
    c, top = m.attn_config(16, hkv, dim, page, m.ATTN_CACHE_E4M3), max(lens)
    ws = torch.empty(m.attn_decode_workspace_size(c, len(lens), nq, top), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    qd, tb, ln, kd, vd, ksd, vsd = R.cuda(q, table, torch.tensor(lens, dtype=torch.int32), kc, vc, ks, vs)
    m.attn_decode(c, len(lens), nq, top, qd, 16 * dim, tb, tb.stride(0), ln, pages, kd, vd, ksd, vsd, dim ** -0.5, out,
                  lse, ws)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        r = slice(b * nq, b * nq + nq)
        ref = R.attend(q[r], R.rows_of(kc, ks, table[b], n), R.rows_of(vc, vs, table[b], n), dim ** -0.5,
                       [n - nq + i + 1 for i in range(nq)])
        R.check_attention(out[r].cpu(), lse[r].cpu(), ref)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens", [[130], [700, 64], [9000]])
@pytest.mark.parametrize("low,high", [(-86, 70), (-89, 100), (-40, 60)])
def test_decode_values_of_very_different_scales(low, high, lens, dim):
    """Rows of values near 2^low before, behind and between rows near 2^high,
    all counting alike: the sums of the probabilities lose none of them."""
    g, page, hkv, nq = rng(dim + high), 16, 2, 2
    table, pages = R.make_table(g, lens, page)
    kc, ks = R.quantised(torch.randn(pages, hkv, page, dim, generator=g))
    v = torch.randn(pages, hkv, page, dim, generator=g)
    exponent = torch.full((pages, hkv, page, 1), float(low))
    for b, n in enumerate(lens):                          # tiles of 64 rows: low, high, low low high and so on
        for j in range((n + page - 1) // page):
            if j // 4 % 3 == 1:
                exponent[table[b, j].long(), :, :] = high
    v = v * torch.exp2(exponent)
    vc, vs = R.quantised(v)
    q = torch.zeros(len(lens) * nq, 16, dim, dtype=torch.bfloat16)
    c, top = m.attn_config(16, hkv, dim, page, m.ATTN_CACHE_E4M3), max(lens)
    ws = torch.empty(m.attn_decode_workspace_size(c, len(lens), nq, top), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    qd, tb, ln, kd, vd, ksd, vsd = R.cuda(q, table, torch.tensor(lens, dtype=torch.int32), kc, vc, ks, vs)
    m.attn_decode(c, len(lens), nq, top, qd, 16 * dim, tb, tb.stride(0), ln, pages, kd, vd, ksd, vsd, dim ** -0.5, out,
                  lse, ws)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        r = slice(b * nq, b * nq + nq)
        ref = R.attend(q[r], R.rows_of(kc, ks, table[b], n), R.rows_of(vc, vs, table[b], n), dim ** -0.5,
                       [n - nq + i + 1 for i in range(nq)])
        R.check_attention(out[r].cpu(), lse[r].cpu(), ref)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("exponent", [-80, -40, 60, 120])
def test_decode_tiny_and_huge_values(exponent, dim):
    """Values down to 2^-80 and up to the largest of bf16 keep their bits: the
    bounds of check_attention in units of 2^exponent."""
    g, page, hkv, nq, lens = rng(dim + exponent), 32, 2, 2, [500, 60]
    table, pages = R.make_table(g, lens, page)
    kc, ks = R.quantised(torch.randn(pages, hkv, page, dim, generator=g))
    vc, vs = R.quantised(torch.randn(pages, hkv, page, dim, generator=g) * 2.0 ** exponent)
    q = (torch.randn(len(lens) * nq, 16, dim, generator=g) * 1.5).bfloat16()
    c, top = m.attn_config(16, hkv, dim, page, m.ATTN_CACHE_E4M3), max(lens)
    ws = torch.empty(m.attn_decode_workspace_size(c, len(lens), nq, top), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    qd, tb, ln, kd, vd, ksd, vsd = R.cuda(q, table, torch.tensor(lens, dtype=torch.int32), kc, vc, ks, vs)
    m.attn_decode(c, len(lens), nq, top, qd, 16 * dim, tb, tb.stride(0), ln, pages, kd, vd, ksd, vsd, dim ** -0.5, out,
                  lse, ws)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        r = slice(b * nq, b * nq + nq)
        o, z, A, big = R.attend(q[r], R.rows_of(kc, ks, table[b], n), R.rows_of(vc, vs, table[b], n), dim ** -0.5,
                                [n - nq + i + 1 for i in range(nq)])
        unit = 2.0 ** -exponent
        R.check_attention(out[r].cpu().double() * unit, lse[r].cpu(), (o * unit, z, A * unit, big))


def test_decode_reports_bad_pages_and_lengths():
    """A bad page reads as zeros (score 0, value 0) and is reported; so is a
    length above max_len (cut) or below zero (none)."""
    for e4m3 in (False, True):
        g = rng(5)
        table, pages = R.make_table(g, [40, 40], 16)
        kc, vc, ks, vs = R.make_cache(g, pages, 1, 16, 64, e4m3)
        c = m.attn_config(2, 1, 64, 16, int(e4m3))
        q = torch.randn(2, 2, 64, generator=g).bfloat16()
        good = table.clone()
        table[0, 1], table[1, 2] = pages, -1
        ws = torch.zeros(m.attn_decode_workspace_size(c, 2, 1, 48), dtype=torch.uint8, device="cuda")
        for tb, lens, cut in ((table, [40, 40], [40, 40]), (good, [60, -3], [48, 0])):
            out = torch.empty(2, 2, 64, dtype=torch.bfloat16, device="cuda")
            err = err_word()
            m.attn_decode(c, 2, 1, 48, q.cuda(), 128, tb.cuda(), 3, torch.tensor(lens, dtype=torch.int32).cuda(),
                          pages, *R.cuda(kc, vc, ks, vs), 0.125, out, None, ws, err=err)
            torch.cuda.synchronize()
            assert err.item() == m.MOE_ERR_BOUNDS
            for b in range(2):
                bad = (tb[b] < 0) | (tb[b] >= pages)
                k, v = (R.rows_of(x, s, torch.where(bad, 0, tb[b]), cut[b]) for x, s in ((kc, ks), (vc, vs)))
                gone = bad[torch.arange(cut[b]) // 16]
                k[gone], v[gone] = 0, 0
                R.check_attention(out[b:b + 1].cpu(), None, R.attend(q[b:b + 1], k, v, 0.125, [cut[b]]))


def test_decode_non_finite_row_reaches_its_own_sequence_only():
    g = rng(6)
    table, pages = R.make_table(g, [100, 100], 32)
    kc, vc, ks, vs = R.make_cache(g, pages, 1, 32, 128, True)
    ks[table[0, 1].long(), 0, 3] = math.nan
    c = m.attn_config(4, 1, 128, 32, 1)
    q = torch.randn(2, 4, 128, generator=g).bfloat16()
    ws = torch.zeros(m.attn_decode_workspace_size(c, 2, 1, 100), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    m.attn_decode(c, 2, 1, 100, q.cuda(), 512, table.cuda(), table.stride(0), torch.tensor([100, 100]).int().cuda(),
                  pages, *R.cuda(kc, vc, ks, vs), 0.1, out, None, ws)
    torch.cuda.synchronize()
    assert out[0].isnan().all() and out[1].isfinite().all()


# ------------------------------------------------------------------ a layer's run


def layer_case(e4m3, dim=128, hq=16, hkv=2, page=32, pages=64):
    g = rng(21)
    inv = torch.pow(10000.0, -torch.arange(0, 64, 2).double() / 64).float()
    qw, kw = ((1 + 0.2 * torch.randn(dim, generator=g)).bfloat16() for _ in range(2))
    L = m.AttentionLayer(hq, hkv, dim, pages, page_size=page, cache_type=int(e4m3), q_weight=qw, k_weight=kw,
                         inv_freq=inv)
    return g, L, qw, kw, inv


def layer_reference(g, L, qkv, qw, kw, inv, pos, e4m3, exact_tail=0):
    """q, and k and v as the cache holds them (the last exact_tail rows as they
    came), of one sequence."""
    c = L.cfg
    (q, _), (k, _), v = R.prepared(qkv, c.q_heads, c.kv_heads, c.head_dim, qw, kw, L.eps, inv, 64, 0, 1.0, pos)
    q, k, v = q.bfloat16(), k.float(), v.float()
    if e4m3:
        k, v = ((x.float() * s[..., None]) for x, s in (R.quantised(k), R.quantised(v)))
    return q, k, v


@pytest.mark.parametrize("e4m3,dim", [(False, 128), (True, 128), (True, 256), (False, 64)])
def test_layer_prompt_chunk_and_steps(e4m3, dim):
    """A prompt, a second chunk after it (read back from the cache), then
    verification rows and single tokens, as a server runs them, of two
    sequences; every output against the whole sequence in 64 bits.  The bound
    adds what rounding q and k once more (bf16) and 8-bit codes that fall to
    the other side of a border may move: 3 % of the largest output."""
    g, L, qw, kw, inv = layer_case(e4m3, dim)
    page, lens = L.cfg.page_size, [200, 77]
    total = 330
    qkv = [torch.randn(total, L.row, generator=g).bfloat16() for _ in lens]
    table = torch.randperm(L.num_pages, generator=g)[:22].view(2, 11).int()
    at = [0, 0]
    got = [[], []]

    def step(counts, fn):
        rows = torch.cat([qkv[b][at[b]:at[b] + n] for b, n in enumerate(counts)]).cuda()
        pos = torch.cat([torch.arange(at[b], at[b] + n) for b, n in enumerate(counts)])
        slots = torch.cat([table[b].long()[torch.arange(at[b], at[b] + n) // page] * page +
                           torch.arange(at[b], at[b] + n) % page for b, n in enumerate(counts)])
        for b, n in enumerate(counts):
            at[b] += n
        out = fn(rows, pos.int().cuda(), slots.int().cuda())
        L.check()
        for b, o in enumerate(out.cpu().split(counts)):
            got[b].append(o)

    step(lens, lambda r, p, s: L.prefill(r, p, s, R.starts(lens).cuda()))
    step([60, 100], lambda r, p, s: L.prefill(r, p, s, R.starts([60, 100]).cuda(), table.cuda(),
                                              R.starts(at).cuda(), sum(at)))
    for nq in (1, 4, 1):
        step([nq, nq], lambda r, p, s: L.decode(r, p, s, table.cuda(), torch.tensor(at).int().cuda(), 352))
    for b in range(2):
        n = at[b]
        out = torch.cat(got[b]).double()
        q, k, v = layer_reference(g, L, qkv[b][:n], qw, kw, inv, torch.arange(n), e4m3)
        o, _, _, _ = R.attend(q, k, v, L.scale, [i + 1 for i in range(n)])
        if e4m3:   # the first prompt saw its own keys before they were rounded to 8 bits
            qe, ke, ve = layer_reference(g, L, qkv[b][:lens[b]], qw, kw, inv, torch.arange(lens[b]), False)
            o[:lens[b]] = R.attend(qe, ke, ve, L.scale, [i + 1 for i in range(lens[b])])[0]
        assert (out - o).abs().max() <= 0.03 * o.abs().max()


def test_layer_decode_captured_and_replayed():
    """The decode calls in a CUDA graph, replayed with new inputs and lengths,
    equal the calls outside it; two graphs in flight on two streams too."""
    g, L, qw, kw, inv = layer_case(True)
    page = L.cfg.page_size
    table = torch.randperm(L.num_pages, generator=g)[:20].view(2, 10).int().cuda()
    L.k_cache.copy_(torch.randn(L.k_cache.shape, generator=g).to(torch.float8_e4m3fn))
    L.v_cache.copy_(torch.randn(L.v_cache.shape, generator=g).to(torch.float8_e4m3fn))
    qkv = torch.randn(2, L.row, generator=g).bfloat16().cuda()
    lens = torch.tensor([100, 250], dtype=torch.int32).cuda()

    def slots():
        p = lens.long() - 1
        return (table.long().gather(1, (p // page)[:, None])[:, 0] * page + p % page).int()

    pos, sl = lens - 1, slots()
    graphs = []
    for _ in range(2):
        L.decode(qkv, pos, sl, table, lens, 320)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = L.decode(qkv, pos, sl, table, lens, 320)
        graphs.append((gr, out))
    for n in ((100, 250), (1, 320), (64, 65)):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        pos.copy_(lens - 1)
        sl.copy_(slots())
        qkv.copy_(torch.randn(2, L.row, generator=g).bfloat16())
        want = L.decode(qkv, pos, sl, table, lens, 320).clone()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for (gr, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
                gr.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out, want)
    L.check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_layer_prompt_captured_and_replayed(e4m3):
    """A prompt's next chunk (write, read-back, attention) in a graph, replayed
    on new rows and lengths of the same sums: what plain calls give."""
    g, L, qw, kw, inv = layer_case(e4m3)
    page = L.cfg.page_size
    table = torch.randperm(L.num_pages, generator=g)[:20].view(2, 10).int().cuda()
    T, total = 37, 300
    qkv = torch.zeros(T, L.row, dtype=torch.bfloat16, device="cuda")
    pos, sl = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))
    cu_q, cu_k = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))

    def fill(new, held):
        p = torch.cat([torch.arange(k - n, k) for n, k in zip(new, held)])
        b = torch.repeat_interleave(torch.arange(2), torch.tensor(new))
        qkv.copy_(torch.randn(T, L.row, generator=g).bfloat16())
        pos.copy_(p.int())
        sl.copy_((table.cpu().long()[b, p // page] * page + p % page).int())
        cu_q.copy_(torch.tensor([0, new[0], T], dtype=torch.int32))
        cu_k.copy_(torch.tensor([0, held[0], total], dtype=torch.int32))

    def call():
        return L.prefill(qkv, pos, sl, cu_q, page_table=table, cu_k=cu_k, total_k=total)

    fill((30, 7), (140, 160))
    call()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = call()
    for new, held in (((30, 7), (140, 160)), ((1, 36), (1, 299)), ((37, 0), (300, 0))):
        fill(new, held)
        gr.replay()
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.isfinite(got.float()).all() and torch.equal(got, call())
    L.check()


def test_layer_refusals():
    _, L, *_ = layer_case(False)
    z = lambda *s, **kw: torch.zeros(*s, **{**dict(dtype=torch.int32, device="cuda"), **kw})  # noqa: E731
    rows = z(4, L.row, dtype=torch.bfloat16)
    ok = (rows, z(4), z(4) - 1)
    with pytest.raises(TypeError, match="qkv"):
        L.prefill(rows.float(), z(4), z(4), z(2))
    with pytest.raises(ValueError, match="qkv must have shape"):
        L.prefill(rows[:, 8:], z(4), z(4), z(2))
    with pytest.raises(ValueError, match="slots must have shape"):
        L.prefill(rows, z(4), z(3), z(2))
    with pytest.raises(ValueError, match="positions is on cpu"):
        L.prefill(rows, z(4).cpu(), z(4), z(2))
    with pytest.raises(TypeError, match="cu_q"):
        L.prefill(*ok, z(2).long())
    with pytest.raises(ValueError, match="total_k"):
        L.prefill(*ok, z(2), z(1, 4), z(2))
    with pytest.raises(ValueError, match="3 sequences"):
        L.decode(*ok, z(3, 4), z(3), 10)
    with pytest.raises(ValueError, match="page_table rows"):
        L.decode(*ok, z(4, 1), z(4), 100)
    with pytest.raises(ValueError, match="no rows"):
        L.prefill(rows[:0], z(0), z(0), z(2))
    L.decode(rows, z(4), z(4) + L.num_pages * 32, z(4, 1), z(4) + 1, 32)
    with pytest.raises(m.MoeError, match="MOE_ERR_BOUNDS"):
        L.check()
    L.check()


def test_layer_prefill_refuses_cached_lengths_without_pages():
    """Without the pages the prefix would be left out with no word of it."""
    _, L, *_ = layer_case(False)
    rows = torch.zeros(4, L.row, dtype=torch.bfloat16, device="cuda")
    z, cu = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for more in (dict(cu_k=cu), dict(total_k=4), dict(cu_k=cu, total_k=4)):
        with pytest.raises(ValueError, match="page_table must be given"):
            L.prefill(rows, z, z - 1, cu, **more)
    L.prefill(rows, z, z - 1, cu)
    L.check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_layer_steps_on_shared_pages(e4m3):
    """One page table row expanded to all sequences (several continuations of
    one prefix): what a table with the row repeated gives, in decode and in a
    prompt's next chunk."""
    g, L, *_ = layer_case(e4m3)
    row = torch.randperm(L.num_pages, generator=g)[:6].int().cuda()
    at = torch.arange(150, device="cuda")
    slots = (row[at // 32] * 32 + at % 32).int()
    L.prefill(torch.randn(150, L.row, generator=g).bfloat16().cuda(), at.int(), slots, R.starts([150]).cuda())
    qkv, pos, none = torch.randn(3, L.row, generator=g).bfloat16().cuda(), torch.full((3,), 150).int().cuda(), torch.full((3,), -1).int().cuda()
    lens = torch.tensor([150, 149, 33], dtype=torch.int32, device="cuda")
    shared, repeated = row[None].expand(3, 6), row[None].repeat(3, 1)
    outs = [L.decode(qkv, pos, none, t, lens, 160) for t in (shared, repeated)]
    assert torch.equal(*outs) and torch.isfinite(outs[0].float()).all()
    cu_q, cu_k = R.starts([1, 1, 1]).cuda(), R.starts([150, 149, 33]).cuda()
    outs = [L.prefill(qkv, pos, none, cu_q, page_table=t, cu_k=cu_k, total_k=332) for t in (shared, repeated)]
    assert torch.equal(*outs) and torch.isfinite(outs[0].float()).all()
    L.check()


def test_layer_check_waits_for_every_stream():
    """An error of a call on another stream, still to run when check() is
    called, is raised by that check and not by a later one."""
    _, L, *_ = layer_case(False)
    rows = torch.zeros(4, L.row, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(4, dtype=torch.int32, device="cuda")
    args = (rows, z, z + L.num_pages * 32, z[:, None].contiguous(), z + 1, 32)
    L.decode(rows, z, z, *args[3:])
    big = torch.zeros(256 << 20, device="cuda")
    L.check()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        for _ in range(60):
            big.add_(1.0)                                    # some 20 ms of work before the call
        L.decode(*args)                                      # slots outside the cache
    with pytest.raises(m.MoeError, match="MOE_ERR_BOUNDS"):
        L.check()
    torch.cuda.synchronize()
    L.check()


# ------------------------------------------------------------------ the binding, streams


def test_binding_refuses_tensors_too_small_for_the_call():
    """What the library would read or write past a tensor's end is refused, as
    are other types and layouts."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    i = lambda *s: z(*s, dt=torch.int32)  # noqa: E731
    f = lambda *s: z(*s, dt=torch.float32)  # noqa: E731
    c = m.attn_config(4, 2, 64, 16, m.ATTN_CACHE_E4M3)
    kc = z(3, 2, 16, 64, dt=torch.uint8)

    def prepare(**kw):
        a = dict(T=4, qkv=z(4, 512), qkv_stride=512, q_weight=z(64), k_weight=z(64), eps=1e-6, inv_freq=f(32),
                 rot_dim=64, rope_layout=0, rope_scale=1.0, positions=i(4), slots=i(4) - 1, num_pages=3, k_cache=kc,
                 v_cache=kc, k_scale=f(3, 2, 16), v_scale=f(3, 2, 16), q_out=z(4, 4, 64), k_out=z(4, 2, 64))
        a.update(kw)
        return m.attn_qkv_prepare(c, *a.values())

    def decode(**kw):
        a = dict(B=2, nq=1, max_len=32, q=z(2, 4, 64), q_stride=256, page_table=i(2, 2), page_table_stride=2,
                 seq_lens=i(2), num_pages=3, k_cache=kc, v_cache=kc, k_scale=f(3, 2, 16), v_scale=f(3, 2, 16),
                 scale=0.1, out=z(2, 4, 64), lse=f(2, 4),
                 ws=z(m.attn_decode_workspace_size(c, 2, 1, 32), dt=torch.uint8))
        a.update(kw)
        return m.attn_decode(c, *a.values())

    def prefill(**kw):
        a = dict(B=1, total_q=4, total_k=6, cu_q=i(2), cu_k=i(2), q=z(4, 4, 64), q_stride=256, k=z(6, 2, 64),
                 k_stride=128, v=z(6, 2, 64), v_stride=128, scale=0.1, causal=True, out=z(4, 4, 64), lse=f(4, 4))
        a.update(kw)
        return m.attn_prefill(c, *a.values())

    def read(**kw):
        a = dict(B=2, total=5, page_table=i(2, 2), page_table_stride=2, cu_lens=i(3), num_pages=3, k_cache=kc,
                 v_cache=kc, k_scale=f(3, 2, 16), v_scale=f(3, 2, 16), k_out=z(5, 2, 64), v_out=z(5, 2, 64))
        a.update(kw)
        return m.attn_kv_read(c, *a.values())

    for call, bad in ((prepare, dict(qkv=z(3, 512))), (prepare, dict(qkv_stride=520)), (prepare, dict(q_weight=z(32))),
                      (prepare, dict(inv_freq=f(16))), (prepare, dict(positions=i(3))), (prepare, dict(slots=i(3))),
                      (prepare, dict(num_pages=4)), (prepare, dict(k_scale=f(3, 2, 8))), (prepare, dict(q_out=z(3, 4, 64))),
                      (prepare, dict(k_out=z(3, 2, 64))), (decode, dict(q=z(1, 4, 64))), (decode, dict(seq_lens=i(1))),
                      (decode, dict(page_table=i(1, 2))), (decode, dict(num_pages=5)), (decode, dict(out=z(1, 4, 64))),
                      (decode, dict(lse=f(4))), (prefill, dict(q=z(3, 4, 64))), (prefill, dict(k=z(5, 2, 64))),
                      (prefill, dict(v_stride=136)), (prefill, dict(cu_q=i(1))), (prefill, dict(out=z(3, 4, 64))),
                      (prefill, dict(lse=f(15))), (read, dict(total=6)), (read, dict(page_table=i(2, 1))),
                      (read, dict(cu_lens=i(2))), (read, dict(v_out=z(4, 2, 64)))):
        with pytest.raises(ValueError, match="may touch"):
            call(**bad)
    with pytest.raises(m.MoeError, match="WORKSPACE"):
        decode(ws=z(128, dt=torch.uint8))
    with pytest.raises(TypeError, match="qkv must be"):
        prepare(qkv=f(4, 512))
    with pytest.raises(TypeError, match="seq_lens must be"):
        decode(seq_lens=i(2).long())
    with pytest.raises(ValueError, match="out must be contiguous"):
        prefill(out=z(4, 64, 4).transpose(1, 2))
    with pytest.raises(ValueError, match="q must be contiguous"):
        prefill(q=z(4, 64, 4).transpose(1, 2))
    assert prepare() == 0 and decode() == 0 and prefill() == 0 and read() == 0
    torch.cuda.synchronize()


def test_calls_follow_their_stream():
    """On a stream other than torch's current one, given or current, the calls
    come after the work before them there."""
    g = rng(31)
    table, pages = R.make_table(g, [300, 77], 16)
    kc, vc, ks, vs = R.make_cache(g, pages, 2, 16, 128, True)
    c = m.attn_config(8, 2, 128, 16, 1)
    q = torch.randn(2, 8, 128, generator=g).bfloat16()
    lens = torch.tensor([300, 77], dtype=torch.int32)
    kd, vd, ksd, vsd, tb, ln, q0 = R.cuda(kc, vc, ks, vs, table, lens, q)
    ws = [torch.empty(m.attn_decode_workspace_size(c, 2, 1, 300), dtype=torch.uint8, device="cuda") for _ in range(2)]
    qd = [torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    outs = [torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    big = torch.zeros(64 << 20, device="cuda")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for n, s in enumerate(streams):
        with torch.cuda.stream(s):
            big.add_(1.0)              # keeps the stream busy before the queries arrive
            qd[n].copy_(q0)
            args = (c, 2, 1, 300, qd[n], 1024, tb, tb.stride(0), ln, pages, kd, vd, ksd, vsd, 0.1, outs[n], None, ws[n])
            if n:
                m.attn_decode(*args)
        if not n:
            m.attn_decode(*args, stream=s)
    torch.cuda.synchronize()
    for b, n in enumerate((300, 77)):
        ref = R.attend(q[b:b + 1], R.rows_of(kc, ks, table[b], n), R.rows_of(vc, vs, table[b], n), 0.1, [n])
        for out in outs:
            R.check_attention(out[b:b + 1].cpu(), None, ref)


@pytest.mark.parametrize("e4m3", [False, True])
def test_cache_offsets_past_32_bits(e4m3):
    """A cache whose last pages lie past 2^32 bytes and elements: written, read
    back and attended to there as at its beginning."""
    hq, hkv, dim, page = 8, 2, 256, 128
    c, pages = m.attn_config(hq, hkv, dim, page, int(e4m3)), (1 << 32) // (hkv * page * dim) + 40
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kc, vc = (torch.empty(pages * hkv * page * dim * (1 if e4m3 else 2), dtype=torch.uint8, device="cuda").view(kind)
              .view(pages, hkv, page, dim) for _ in "kv")
    ks, vs = (torch.empty(pages, hkv, page, device="cuda") if e4m3 else None for _ in "kv")
    g, lens, err = rng(9), [700, 300], err_word()
    T = sum(lens)
    qkv = torch.randn(T, (hq + 2 * hkv) * dim, generator=g).bfloat16().cuda()
    results = []
    for first in (3, pages - 12):
        table = (first + torch.randperm(12, generator=rng(4))[:9].int()).cuda()
        rows = [table[:6], table[6:]]
        slots = torch.cat([(r.long()[torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page).int()
                           for r, n in zip(rows, lens)])
        q = torch.empty(T, hq, dim, dtype=torch.bfloat16, device="cuda")
        m.attn_qkv_prepare(c, T, qkv, qkv.stride(0), None, None, 0.0, None, 0, 0, 1.0, None, slots, pages, kc, vc, ks, vs, q,
                           None, err=err)
        tb = torch.zeros(2, 6, dtype=torch.int32, device="cuda")
        tb[0], tb[1, :3] = rows[0], rows[1]
        k, v = (torch.empty(T, hkv, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        m.attn_kv_read(c, 2, T, tb, 6, R.starts(lens).cuda(), pages, kc, vc, ks, vs, k, v, err=err)
        last = q[torch.tensor([lens[0] - 1, T - 1], device="cuda")]
        out, ws = torch.empty_like(last), torch.empty(m.attn_decode_workspace_size(c, 2, 1, 700), dtype=torch.uint8, device="cuda")
        m.attn_decode(c, 2, 1, 700, last, hq * dim, tb, 6, torch.tensor(lens, dtype=torch.int32, device="cuda"), pages, kc, vc,
                      ks, vs, dim ** -0.5, out, None, ws, err=err)
        torch.cuda.synchronize()
        assert err.item() == 0
        results.append((k, v, out))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    k, v, out = (t.cpu() for t in results[1])
    x = qkv.cpu().view(T, hq + 2 * hkv, dim).float()
    for got, ref in ((k, x[:, hq:hq + hkv]), (v, x[:, hq + hkv:])):
        if e4m3:
            codes, scale = R.quantised(ref)
            ref = codes.float() * scale[..., None]
        assert ((got.double() - ref.double()).abs() <= 2.0 ** -8 * ref.double().abs() * 1.001 + 1e-30).all()
    for b, s in enumerate((slice(0, 700), slice(700, 1000))):
        ref = R.attend(x[s][-1:, :hq], k[s], v[s], dim ** -0.5, [lens[b]])
        # the rows read back were rounded once more to bf16: 2^-8 of scores' and values' sizes
        assert ((out[b:b + 1].double() - ref[0]).abs() <= (2.0 ** -6 + 2.0 ** -8 * 2 * ref[3][..., None]) * ref[2]).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prefill_offsets_past_32_bits(dim):
    """Packed rows past 2^32 elements of q and out, 2^31 of k and v: the same
    bits as the same sequence at the beginning."""
    hq, hkv, n = 4, 2, 300
    far = (1 << 32) // (hq * dim) + 1000
    q = torch.empty(far + n, hq, dim, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty(far + n, hkv, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    g = rng(dim)
    for t in (q, k, v):
        t[:n] = torch.randn(n, *t.shape[1:], generator=g).bfloat16()
        t[far:] = t[:n]
    out = torch.empty(far + n, hq, dim, dtype=torch.bfloat16, device="cuda")
    lse, c, err = torch.empty(far + n, hq, device="cuda"), m.attn_config(hq, hkv, dim), err_word()
    for first in (0, far):
        cu = torch.tensor([first, first + n], dtype=torch.int32, device="cuda")
        m.attn_prefill(c, 1, far + n, far + n, cu, cu, q, hq * dim, k, hkv * dim, v, hkv * dim, dim ** -0.5, True, out, lse,
                       err=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(out[:n], out[far:]) and torch.equal(lse[:n], lse[far:])
    R.check_attention(out[far:].cpu(), lse[far:].cpu(),
                      R.attend(q[:n].cpu(), k[:n].cpu(), v[:n].cpu(), dim ** -0.5, prefill_limit(n, n, True)))


def test_all_calls_at_once():
    """Prompts of every head size, decode over both caches, writes and
    read-backs on streams of their own at the same time: what each gives alone."""
    def prompt(dim, hq, hkv, lens):
        g = rng(dim + hq)
        q, k, v = (torch.randn(sum(lens), h, dim, generator=g).bfloat16().cuda() for h in (hq, hkv, hkv))
        cu, c = R.starts(lens).cuda(), m.attn_config(hq, hkv, dim)

        def call(out):
            m.attn_prefill(c, len(lens), q.shape[0], q.shape[0], cu, cu, q, hq * dim, k, hkv * dim, v, hkv * dim, dim ** -0.5,
                           True, out[0], out[1])
        return call, [(q.shape, torch.bfloat16), (q.shape[:2], torch.float32)]

    def steps(dim, e4m3, lens, nq):
        g, hkv, page = rng(dim + nq), 2, 32
        table, pages = R.make_table(g, lens, page)
        kd, vd, ksd, vsd = R.cuda(*R.make_cache(g, pages, hkv, page, dim, e4m3))
        q = torch.randn(len(lens) * nq, 16, dim, generator=g).bfloat16().cuda()
        c, top = m.attn_config(16, hkv, dim, page, int(e4m3)), max(lens)
        tb, ln = R.cuda(table, torch.tensor(lens, dtype=torch.int32))
        ws = torch.empty(m.attn_decode_workspace_size(c, len(lens), nq, top), dtype=torch.uint8, device="cuda")
        total, cu = sum(lens), R.starts(lens).cuda()

        def call(out):
            m.attn_decode(c, len(lens), nq, top, q, 16 * dim, tb, tb.stride(0), ln, pages, kd, vd, ksd, vsd, dim ** -0.5,
                          out[0], out[1], ws)
            m.attn_kv_read(c, len(lens), total, tb, tb.stride(0), cu, pages, kd, vd, ksd, vsd, out[2], out[3])
        return call, [(q.shape, torch.bfloat16), (q.shape[:2], torch.float32)] + 2 * [((total, hkv, dim), torch.bfloat16)]

    jobs = [prompt(256, 16, 2, [300, 700]), prompt(128, 16, 16, [600, 1, 90]), prompt(64, 12, 4, [513]),
            prompt(256, 48, 48, [200, 129]), steps(128, True, [3000, 20, 900], 4), steps(256, False, [77, 2000], 1),
            steps(64, True, [500] * 40, 8)]
    fresh = lambda kinds: [torch.full(s, math.nan, dtype=t, device="cuda") for s, t in kinds]  # noqa: E731
    alone, rounds, streams = [], [], [torch.cuda.Stream() for _ in jobs]
    for call, kinds in jobs:
        alone.append(fresh(kinds))
        call(alone[-1])
        torch.cuda.synchronize()
    for _ in range(8):
        rounds.append([fresh(kinds) for _, kinds in jobs])
    torch.cuda.synchronize()
    for outs in rounds:
        for (call, _), out, s in zip(jobs, outs, streams):
            with torch.cuda.stream(s):
                call(out)
    torch.cuda.synchronize()
    for outs in rounds:
        for out, want in zip(outs, alone):
            assert all(torch.equal(a, b) and torch.isfinite(b.float()).all() for a, b in zip(out, want))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prefill_captured_and_replayed_twice_at_once(dim):
    """Two graphs that hold the call, replayed on two streams at the same time
    with lengths that changed since the capture."""
    hq, hkv, T, g = 16, 4, 700, rng(dim)
    q, k, v = (torch.randn(T, h, dim, generator=g).bfloat16().cuda() for h in (hq, hkv, hkv))
    cu, c = R.starts([300, 400]).cuda(), m.attn_config(hq, hkv, dim)
    outs = [torch.zeros(T, hq, dim, dtype=torch.bfloat16, device="cuda") for _ in range(3)]

    def call(out):
        m.attn_prefill(c, 2, T, T, cu, cu, q, hq * dim, k, hkv * dim, v, hkv * dim, dim ** -0.5, True, out)

    call(outs[2])
    torch.cuda.synchronize()
    graphs = []
    for out in outs[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(out)
    streams = [torch.cuda.Stream() for _ in graphs]
    for lens in ([300, 400], [1, 699], [700, 0], [555, 145]):
        cu.copy_(R.starts(lens))
        call(outs[2])
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])
        R.check_attention(outs[2][:lens[0]].cpu(), None, R.attend(q[:lens[0]].cpu(), k[:lens[0]].cpu(), v[:lens[0]].cpu(),
                                                                  dim ** -0.5, prefill_limit(lens[0], lens[0], True)))


@pytest.mark.parametrize("side", ["q", "k"])
@pytest.mark.parametrize("layout", [0, 1])
def test_prepare_with_one_side_normalised(side, layout):
    T, hq, hkv, dim, page = 70, 6, 2, 128, 16
    c = m.attn_config(hq, hkv, dim, page, m.ATTN_CACHE_E4M3)
    d = prepare_case(T, hq, hkv, dim, 96, layout, True, page, 5)
    d["kw" if side == "q" else "qw"] = None
    check_prepared(c, d, T, 96, layout, run_prepare(c, d, T, 96, layout))


def test_prefill_most_sequences():
    """65535 sequences, most of them empty, some past the 64000th not."""
    g, B, hq, hkv, dim = rng(3), 65535, 2, 1, 64
    lens = [0] * B
    for b in [0, 5, 639, 640, 641, 30000, 64001, 65534] + torch.randint(0, B, (1500,), generator=g).tolist():
        lens[b] = 1 + b % 3 + (b % 640 == 0) * 150
    cu = R.starts(lens)
    T = sum(lens)
    q, k, v = (torch.randn(T, h, dim, generator=g).bfloat16() for h in (hq, hkv, hkv))
    qd, kd, vd, cd = R.cuda(q, k, v, cu)
    out, lse, err = torch.full_like(qd, math.nan), torch.full((T, hq), math.nan, device="cuda"), err_word()
    m.attn_prefill(m.attn_config(hq, hkv, dim), B, T, T, cd, cd, qd, hq * dim, kd, hkv * dim, vd, hkv * dim, 0.125, True, out,
                   lse, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    out, lse = out.cpu(), lse.cpu()
    for b in [i for i, n in enumerate(lens) if n]:
        r = slice(cu[b], cu[b + 1])
        R.check_attention(out[r], lse[r], R.attend(q[r], k[r], v[r], 0.125, prefill_limit(lens[b], lens[b], True)))


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_most_sequences_with_strided_queries(e4m3):
    """65535 sequences of up to 40 rows, pages shared, query rows and page
    tables wider than what the call reads."""
    g, B, hq, hkv, dim, page, pages = rng(4), 65535, 2, 1, 64, 16, 50
    kc, vc, ks, vs = R.make_cache(g, pages, hkv, page, dim, e4m3)
    lens = torch.randint(0, 41, (B,), generator=g).int()
    table = torch.randint(0, pages, (B, 5), generator=g).int()
    q = torch.randn(B, hq * dim + 24, generator=g).bfloat16()
    c = m.attn_config(hq, hkv, dim, page, int(e4m3))
    qd, tb, ln, kd, vd, ksd, vsd = R.cuda(q, table, lens, kc, vc, ks, vs)
    ws = torch.empty(m.attn_decode_workspace_size(c, B, 1, 40), dtype=torch.uint8, device="cuda")
    out, lse, err = torch.full((B, hq, dim), math.nan, dtype=torch.bfloat16, device="cuda"), torch.empty(B, hq, device="cuda"), err_word()
    m.attn_decode(c, B, 1, 40, qd, q.shape[1], tb, 5, ln, pages, kd, vd, ksd, vsd, 0.125, out, lse, ws, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    out, lse = out.cpu(), lse.cpu()
    assert torch.isfinite(out.float()).all() and torch.equal(lse.isinf().all(1), lens == 0)
    for b in [0, 1, 383, 384, 511, 512, B - 1] + torch.randint(0, B, (600,), generator=g).tolist():
        n = int(lens[b])
        ref = R.attend(q[b:b + 1, :hq * dim].view(1, hq, dim), R.rows_of(kc, ks, table[b], n), R.rows_of(vc, vs, table[b], n),
                       0.125, [n])
        R.check_attention(out[b:b + 1], lse[b:b + 1], ref)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_longest_sequence(e4m3):
    """2^30 rows, the most that a call takes, beside a short sequence: a page
    table of 2^23 entries over four pages.  All keys count alike, so the output is
    the mean of the pages' values, each of which counts equally often."""
    g, hkv, dim, page = rng(5), 1, 64, 128
    n = 1 << 30
    kc, vc, ks, vs = R.make_cache(g, 4, hkv, page, dim, e4m3)
    c = m.attn_config(2, hkv, dim, page, int(e4m3))
    table = (torch.arange(2 * (n // page), device="cuda", dtype=torch.int32) % 4).view(2, -1)
    lens = torch.tensor([n, 512], dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 2, dim, dtype=torch.bfloat16, device="cuda")
    kd, vd, ksd, vsd = R.cuda(kc, vc, ks, vs)
    ws = torch.empty(m.attn_decode_workspace_size(c, 2, 1, n), dtype=torch.uint8, device="cuda")
    out, lse, err = torch.empty_like(q), torch.empty(2, 2, device="cuda"), err_word()
    m.attn_decode(c, 2, 1, n, q, 2 * dim, table, table.stride(0), lens, 4, kd, vd, ksd, vsd, 0.125, out, lse, ws, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    values = R.rows_of(vc, vs, torch.arange(4), 512)[:, 0]
    mean, size = values.mean(0), values.abs().mean(0)
    # 2^30 terms over 148 blocks, two or three groups and 16 lanes: 2^17 additions a sum of l, 2^17 products of 64 keys a sum
    # of the output, each off by half a step of what has come together: 2^17 2^-24 = 2^-7 at the worst, all to one side
    for b, tol in ((0, 2.0 ** -7 + 2.0 ** -8), (1, 2.0 ** -8 + 2.0 ** -12)):
        assert ((out[b].cpu().double() - mean).abs() <= 2.0 ** -8 * mean.abs() + tol * size).all()
    assert abs(lse[0, 0].item() - math.log(n)) <= 2.0 ** -7 and abs(lse[1, 0].item() - math.log(512)) <= 2.0 ** -12
