"""The 8-bit paged cache on the GPU against plain implementations
(tests/kv8_ref.py): append, attention, and a run of both as a decode loop
uses them."""
import numpy as np
import pytest
import torch

from kv_cache_decode_dualcache_b200 import build, fdllm
from tests import kv8_ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    require_gpu()
    build.build()


def _gpu(cache):
    d = {n: t.cuda() for n, t in cache.items()}
    return d, fdllm.Kv8Cache(d["k"], d["v"], d["k_scale"], d["v_scale"], d["table"])


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(rows):
    return [int(x) for x in np.concatenate([[0], np.cumsum(rows)])]


def _check_attention(cache, q, starts, lens, scale, got, sentinel=None):
    want, *sizes = kv8_ref.attention(cache, q, starts, lens, scale)
    got = got.cpu()
    live = torch.zeros(q.shape[0], dtype=torch.bool)
    live[starts[0]:starts[-1]] = True
    if sentinel is not None:
        assert (got[~live] == sentinel).all(), "rows behind the last sequence were written"
    tol = kv8_ref.attention_tol(*sizes, want, max(lens + [1]), q.shape[2], q.dtype)
    got, want, tol = got.double()[live], want[live], tol[live]
    # a result beyond the type's largest number rounds to infinity
    big = want.abs() > torch.finfo(q.dtype).max
    bad = int((got[big] != torch.sign(want[big]) * float("inf")).sum())
    assert bad == 0 and bool(torch.isfinite(got[~big]).all()), "not finite"
    over = (got - want).abs()[~big] / tol[~big]
    assert bool((over <= 1).all()), (int((over > 1).sum()), float(over.max()))


HEADS = [(4, 4, 32), (8, 2, 64), (8, 8, 128), (28, 4, 128), (16, 1, 128), (6, 2, 32)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv,hd", HEADS)
@pytest.mark.parametrize("rows,lens", [
    ([1], [1]),                                  # one token, itself
    ([1, 1, 1, 1, 1], [0, 15, 16, 17, 511]),     # no keys; around a scale block
    ([32], [577]),                               # a diffusion block
    ([3, 0, 17, 1], [63, 64, 65, 1300]),         # pages, an idle slot
    ([70], [129]),                               # several row tiles
    ([8, 2, 40], [700, 0, 128]),                 # up to 64 and 128 rows a K/V head
    ([150], [333]),                              # prompt-sized
])
def test_attention(dtype, hq, hkv, hd, rows, lens):
    g = torch.Generator().manual_seed(sum(rows) + 7 * sum(lens) + hq + hd)
    cache = kv8_ref.make_cache(g, lens, hkv, hd)
    T = sum(rows)
    q = (2 * torch.randn(T + 3, hq, hd, generator=g)).to(TYPES[dtype])
    starts = _starts(rows)
    _, c = _gpu(cache)
    out = torch.full((T + 3, hq, hd), 7.0, dtype=q.dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fdllm.fdllm_kv8_attention(c, q.cuda(), _i32(starts), _i32(lens), out=out, status=status)
    assert status.item() == 0
    _check_attention(cache, q, starts, lens, hd ** -0.5, out, sentinel=7.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("max_q,max_len,space", [(0, 0, True), (1, 1, True), (40, 5000, True),
                                                  (0, 0, False)])
def test_attention_hints_and_workspace_do_not_change_results(dtype, max_q, max_len, space):
    """Wrong launch hints, and no workspace at all, only cost time."""
    g = torch.Generator().manual_seed(5)
    rows, lens = [9, 40, 1], [3000, 1025, 4999]
    cache = kv8_ref.make_cache(g, lens, 2, 64, extra_width=9)
    q = torch.randn(sum(rows), 8, 64, generator=g).to(TYPES[dtype])
    starts = _starts(rows)
    _, c = _gpu(cache)
    ws = None if space else torch.empty(0, dtype=torch.uint8, device="cuda")
    got = fdllm.fdllm_kv8_attention(c, q.cuda(), _i32(starts), _i32(lens), scale=0.2, max_q=max_q,
                                    max_len=max_len, workspace=ws)
    _check_attention(cache, q, starts, lens, 0.2, got)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv,hd", HEADS)
@pytest.mark.parametrize("rows,lens", [
    ([17], [1]), ([32], [577]), ([3, 0, 17, 1], [63, 64, 65, 1300]), ([70], [129]),
    ([8, 2, 40], [700, 0, 128]), ([150, 33], [333, 2000])])
def test_attention_where_contexts_may_be_long(dtype, hq, hkv, hd, rows, lens):
    """Page tables for a million tokens, of which the sequences use little:
    the call is laid out for long contexts."""
    g = torch.Generator().manual_seed(sum(rows) + 5 * sum(lens) + hq + hd)
    cache = kv8_ref.make_cache(g, lens, hkv, hd)
    T = sum(rows)
    q = (2 * torch.randn(T + 3, hq, hd, generator=g)).to(TYPES[dtype])
    starts = _starts(rows)
    d, _ = _gpu(cache)
    table = torch.full((len(lens), 16384), -1, dtype=torch.int32, device="cuda")
    table[:, :d["table"].shape[1]] = d["table"]
    c = fdllm.Kv8Cache(d["k"], d["v"], d["k_scale"], d["v_scale"], table)
    out = torch.full((T + 3, hq, hd), 7.0, dtype=q.dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fdllm.fdllm_kv8_attention(c, q.cuda(), _i32(starts), _i32(lens), out=out, status=status)
    assert status.item() == 0
    _check_attention(cache, q, starts, lens, hd ** -0.5, out, sentinel=7.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv,hd,most", [(8, 2, 64, 1), (28, 4, 128, 1), (28, 4, 128, 17), (8, 2, 64, 33)])
@pytest.mark.parametrize("n", [33, 64, 100])
def test_attention_many_sequences(dtype, n, hq, hkv, hd, most):
    """More sequences than a warp scans at once, idle slots among them, split runs
    in the first, the 33rd and later ones."""
    g = torch.Generator().manual_seed(n + most)
    lens = [int(x) for x in torch.randint(0, 300, (n,), generator=g)]
    rows = [int(x) for x in torch.randint(0, most + 1, (n,), generator=g)]
    for i, x in ((0, 1900), (32, 2500), (n - 1, 3000), (n // 2, 0)):
        lens[i], rows[i] = x, most
    starts = _starts(rows)
    cache = kv8_ref.make_cache(g, lens, hkv, hd)
    q = torch.randn(sum(rows) + 2, hq, hd, generator=g).to(TYPES[dtype])
    _, c = _gpu(cache)
    for kw in ({}, dict(max_q=most, max_len=3000)):
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        fdllm.fdllm_kv8_attention(c, q.cuda(), _i32(starts), _i32(lens), out=out, status=status, **kw)
        assert status.item() == 0
        _check_attention(cache, q, starts, lens, hd ** -0.5, out, sentinel=7.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_strided_rows_and_starts_offset(dtype):
    """q is a slice of a fused projection, out a slice of a wider buffer, the
    first sequence does not start at row 0."""
    g = torch.Generator().manual_seed(6)
    rows, lens = [5, 33], [200, 90]
    cache = kv8_ref.make_cache(g, lens, 2, 128)
    qkv = torch.randn(44, 6 + 4, 128, generator=g).to(TYPES[dtype])
    starts = [4, 9, 42]
    _, c = _gpu(cache)
    wide = torch.full((44, 2, 6, 128), 7.0, dtype=qkv.dtype, device="cuda")
    fdllm.fdllm_kv8_attention(c, qkv.cuda()[:, :6], _i32(starts), _i32(lens), out=wide[:, 1])
    _check_attention(cache, qkv[:, :6], starts, lens, 128 ** -0.5, wide[:, 1], sentinel=7.0)
    assert (wide[:, 0] == 7.0).all()


def test_attention_peaked_and_uneven_scales():
    """Scores of several hundred, value scales over 2^-60 .. 2^20 (the heavy
    token's is the smallest), an all-zero block and a negative softmax scale."""
    g = torch.Generator().manual_seed(7)
    lens, rows = [300], [4]
    for dtype in TYPES.values():
        for scale in (3.0, -1.0, 0.0):
            cache = kv8_ref.make_cache(g, lens, 1, 64)
            pages = cache["table"][0, :5].long()
            vs = torch.exp2(torch.linspace(-60, 20, 20)[torch.randperm(20, generator=g)])
            cache["v_scale"][pages, 0] = vs.view(5, 4)
            cache["v_scale"][pages[1], 0, 2] = 0.0
            cache["v"][pages[1], 0, 32:48] = 0
            cache["k_scale"][pages[2], 0, 1] = 0.0
            q = torch.randn(4, 2, 64, generator=g).to(dtype)
            _, c = _gpu(cache)
            got = fdllm.fdllm_kv8_attention(c, q.cuda(), _i32([0, 4]), _i32(lens), scale=scale)
            _check_attention(cache, q, [0, 4], lens, scale, got)


@pytest.mark.parametrize("space", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
def test_attention_value_scales_just_below_a_power_of_two(dtype, space):
    """Equal scores, value scales 1 and then 2^8 (1 - 2^-15) or so: the later
    keys' weights pass the first reference by almost as much as it may be passed
    before it moves, times a mantissa of almost 2.  The results are finite."""
    g = torch.Generator().manual_seed(16)
    for late in (255.99, 127.995, 2.0 - 2.0 ** -20, 511.98):
        lens, hd = [192], 64
        cache = kv8_ref.make_cache(g, lens, 1, hd)
        pages = cache["table"][0, :3].long()
        cache["v_scale"][pages] = 1.0
        cache["v_scale"][pages[2], 0, :2] = late       # keys 128 .. 159
        for q in (torch.zeros(3, 2, hd), torch.randn(3, 2, hd, generator=g) * 1e-3):
            q = q.to(TYPES[dtype])
            _, c = _gpu(cache)
            ws = None if space else torch.empty(0, dtype=torch.uint8, device="cuda")
            got = fdllm.fdllm_kv8_attention(c, q.cuda(), _i32([0, 3]), _i32(lens), workspace=ws)
            _check_attention(cache, q, [0, 3], lens, hd ** -0.5, got)


@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("dtype", TYPES)
def test_attention_scores_beyond_2_24(dtype, rows):
    """Scores up to 2^30 and down to -2^30, whose neighbours in float32 are up to 128
    apart: finite weights all the same.  With one key, or two that are equal, the
    result is the value: the weight and its sum are off by at most 2^-11 (one fp16
    term) and 2^-20 (exp2, the sums, the division)."""
    hd = 64
    cache = kv8_ref.make_cache(torch.Generator().manual_seed(18), [2], 1, hd)
    page = int(cache["table"][0, 0])
    cache["k"][page, 0] = 64
    cache["k_scale"][page, 0, 0] = 2.0 ** -6
    cache["v"][page, 0, 1] = cache["v"][page, 0, 0]
    for vs in (1.0, 1.75):
        cache["v_scale"][page, 0, 0] = vs
        _, c = _gpu(cache)
        v = cache["v"][page, 0, 0].double() * vs
        tol = v.abs() * (2.0 ** -11 + 2.0 ** -20 + torch.finfo(TYPES[dtype]).eps / 2)
        for n in (1, 2):
            for sign in (1, -1):
                for e in range(20, 31):
                    for m in (1.0, 1.13, 1.31, 1.5, 1.77, 1.93):
                        # q . k = hd, so the score in base 2 is sign m 2^e or so
                        scale = sign * m * 2.0 ** e / hd / 1.4426950408889634
                        q = torch.ones(rows, 1, hd, dtype=TYPES[dtype], device="cuda")
                        got = fdllm.fdllm_kv8_attention(c, q, _i32([0, rows]), _i32([n]), scale=scale)
                        assert ((got.cpu().double() - v).abs() <= tol).all(), (vs, n, sign, e, m)


@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("dtype", TYPES)
def test_attention_large_scores_step_by_a_power_of_two(dtype, rows):
    """Equal scores of 2^22 to 2^29, value scales 1 and then 2^6 to 2^9: where
    float32 has no number between, a later key passes the reference by just what
    it may, or by the next number."""
    hd, lens = 64, [192]
    cache = kv8_ref.make_cache(torch.Generator().manual_seed(19), lens, 1, hd)
    pages = cache["table"][0, :3].long()
    cache["k"][pages] = 64
    cache["k_scale"][pages] = 2.0 ** -6
    q = torch.ones(rows, 1, hd, dtype=TYPES[dtype])
    for up in (6, 7, 8, 9):
        cache["v_scale"][pages] = 1.0
        cache["v_scale"][pages[2]] = 2.0 ** up * 0.99999
        _, c = _gpu(cache)
        for sign in (1, -1):
            for e in range(22, 30):
                for m in (1.0, 1.2500001, 1.5000002, 1.9):
                    scale = sign * m * 2.0 ** e / hd / 1.4426950408889634
                    for space in (None, torch.empty(0, dtype=torch.uint8, device="cuda")):
                        got = fdllm.fdllm_kv8_attention(c, q.cuda(), _i32([0, rows]), _i32(lens), scale=scale,
                                                        workspace=space)
                        assert torch.isfinite(got).all(), (up, sign, e, m)


def test_attention_uses_the_codes_full_range():
    """A code of -128 (not one the append writes) reads as -128."""
    cache = kv8_ref.make_cache(torch.Generator().manual_seed(0), [1], 1, 32)
    page = int(cache["table"][0, 0])
    cache["v"][page, 0, 0] = torch.arange(-128, 128, 8).to(torch.int8)
    cache["v_scale"][page, 0, 0] = 0.5
    _, c = _gpu(cache)
    got = fdllm.fdllm_kv8_attention(c, torch.ones(1, 1, 32, device="cuda"), _i32([0, 1]), _i32([1]))
    assert torch.equal(got.cpu()[0, 0], torch.arange(-128, 128, 8) * 0.5)


def test_attention_bad_pages_and_lengths_are_reported():
    """Page ids outside the pool leave their keys out; a length beyond the
    table is cut."""
    g = torch.Generator().manual_seed(8)
    lens = [200, 70]
    cache = kv8_ref.make_cache(g, lens, 2, 64, extra_width=0)
    q = torch.randn(2, 4, 64, generator=g)
    for bad in (-1, 1 << 30, cache["k"].shape[0]):
        d, c = _gpu(cache)
        d["table"][0, 1] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = fdllm.fdllm_kv8_attention(c, q.cuda(), _i32([0, 1, 2]), _i32(lens), status=status)
        assert status.item() == fdllm.KV8_BAD_PAGE
        # the same as if the sequence consisted of its other pages' keys
        k, v = (kv8_ref.dense(cache, w, 0, 200) for w in "kv")
        k, v = (torch.cat([x[:, :64], x[:, 128:]], 1) for x in (k, v))
        x = q[0].double().view(2, 2, 64)
        p = torch.softmax(torch.einsum("grd,gld->grl", x, k) / 8, -1)
        want = torch.einsum("grl,gld->grd", p, v).reshape(4, 64)
        assert (got[0].cpu().double() - want).abs().max() < 1e-5 * want.abs().max()
    d, c = _gpu(cache)
    status.zero_()
    got = fdllm.fdllm_kv8_attention(c, q.cuda(), _i32([0, 1, 2]), _i32([200, -5]), status=status)
    assert status.item() == fdllm.KV8_BAD_RANGE and (got[1] == 0).all()
    # starts that run backwards or past the rows are clamped, nothing else is touched
    out = torch.full((2, 4, 64), 7.0, device="cuda")
    fdllm.fdllm_kv8_attention(c, q.cuda(), _i32([1, 0, 99]), _i32(lens), out=out)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("starts,bad", [([0, 1, 2], False), ([0, 0, 0], False), ([2, 2, 2], False), ([1, 0, 2], True),
                                        ([0, 1, 3], True), ([-1, 1, 2], True), ([3, 3, 3], True), ([0, 5, 2], True)])
@pytest.mark.parametrize("rows", [2, 140])
def test_starts_out_of_range_are_reported(starts, bad, rows):
    """By both calls (and both attention kernels); the starts are clamped, rows of
    no sequence are left as they are."""
    g = torch.Generator().manual_seed(20)
    cache = kv8_ref.make_cache(g, [200, 70], 2, 64)
    d, c = _gpu(cache)
    q = torch.randn(rows, 4, 64, generator=g).to(torch.float16).cuda()
    # 1 stands for the middle, 2 for the end, 3 and 5 for what is behind it
    at = _i32([x if x < 1 else rows // 2 if x == 1 else rows + x - 2 for x in starts])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((rows, 4, 64), 7.0, dtype=q.dtype, device="cuda")
    fdllm.fdllm_kv8_attention(c, q, at, _i32([130, 70]), out=out, status=st)
    assert st.item() == (fdllm.KV8_BAD_RANGE if bad else 0) and torch.isfinite(out).all()
    if starts in ([0, 0, 0], [2, 2, 2], [3, 3, 3]):
        assert (out == 7.0).all()
    st.zero_()
    fdllm.fdllm_kv8_append(c, q[:, :2], q[:, 2:], at, _i32([0, 0]), status=st)
    assert st.item() & fdllm.KV8_BAD_RANGE == (fdllm.KV8_BAD_RANGE if bad else 0)


def test_a_cache_keeps_its_tensors():
    """The C struct holds their addresses: a table assigned later (a longer one,
    say) would not be seen, and the old one's memory be read when it is gone."""
    d, c = _gpu(kv8_ref.make_cache(torch.Generator().manual_seed(0), [70], 1, 64))
    for name in ("k", "v", "k_scale", "v_scale", "page_table", "n_seqs", "struct", "address"):
        with pytest.raises(AttributeError, match="read-only"):
            setattr(c, name, getattr(c, name))
    assert c.page_table.data_ptr() == c.struct.page_table == d["table"].data_ptr()


def test_attention_refuses_a_small_workspace():
    cache = kv8_ref.make_cache(torch.Generator().manual_seed(0), [9000], 1, 64)
    _, c = _gpu(cache)
    q = torch.zeros(1, 1, 64, device="cuda")
    need = fdllm.fdllm_kv8_attention_workspace(c, 1, 1, q.dtype, 0, 9000)
    assert need > 0
    with pytest.raises(fdllm.FdllmError) as e:
        fdllm.fdllm_kv8_attention(c, q, _i32([0, 1]), _i32([9000]), max_len=9000,
                                  workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.code == fdllm.FDLLM_ERR_ARG and str(need) in str(e.value)


def test_offsets_beyond_32_bits():
    """Pages of one layer inside a pool of all layers: page strides of 1 MiB,
    pages beyond byte 2^32; K and V of a page side by side."""
    g = torch.Generator().manual_seed(9)
    pages, hkv, hd = 4200, 2, 128
    small = kv8_ref.make_cache(g, [250, 130], hkv, hd, spare=0)
    n = small["k"].shape[0]
    pool = torch.zeros(pages, 1 << 20, dtype=torch.int8, device="cuda")
    block = hkv * 64 * hd
    k = pool[:, :block].view(pages, hkv, 64, hd)
    v = pool[:, block:2 * block].view(pages, hkv, 64, hd)
    scales = torch.zeros(pages, 2, hkv, 4, device="cuda")
    far = torch.tensor([4199 - 7 * i for i in range(n)])
    k[far.cuda()], v[far.cuda()] = small["k"].cuda(), small["v"].cuda()
    scales[far.cuda(), 0], scales[far.cuda(), 1] = small["k_scale"].cuda(), small["v_scale"].cuda()
    table = small["table"].clone()
    ok = (table >= 0) & (table < n)
    table[ok] = far[table[ok].long()].to(torch.int32)
    c = fdllm.Kv8Cache(k, v, scales[:, 0], scales[:, 1], table.cuda())
    q = torch.randn(2, 4, hd, generator=g).to(torch.bfloat16)
    lens = [250, 130]
    got = fdllm.fdllm_kv8_attention(c, q.cuda(), _i32([0, 1, 2]), _i32(lens))
    _check_attention(small, q, [0, 1, 2], lens, hd ** -0.5, got)
    x = torch.randn(2, hkv, hd, generator=g).to(torch.bfloat16)
    fdllm.fdllm_kv8_append(c, x.cuda(), x.cuda(), _i32([0, 1, 2]), _i32(lens))
    ref = {a: b.clone() for a, b in small.items()}
    kv8_ref.append(ref, x, x, [0, 1, 2], lens)
    assert torch.equal(k[far.cuda()].cpu(), ref["k"]) and torch.equal(v[far.cuda()].cpu(), ref["v"])


# ------------------------------------------------------------------ append
def _rope(n, hd, theta=1e4):
    a = torch.arange(n, dtype=torch.float64)[:, None] * theta ** (
        -2.0 * torch.arange(hd // 2, dtype=torch.float64) / hd)
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _check_append(cache, c_gpu, got, ref, status, lens_out):
    """Codes, scales and outputs to the bit (NaN where nothing was written)."""
    assert status.item() == 0
    for n in ("k", "v"):
        assert torch.equal(c_gpu[n].cpu(), cache[n]), n
    for n in ("k_scale", "v_scale"):
        assert torch.equal(c_gpu[n].cpu().nan_to_num(nan=-1.0), cache[n].nan_to_num(nan=-1.0)), n
    for x, w in zip(got, (ref["q"], ref["k"], ref["v"])):
        if w is not None and x is not None:
            live = ~w.isnan().flatten(1).all(1)
            assert torch.equal(x.cpu()[live].nan_to_num(), w[live].nan_to_num())
    assert lens_out.tolist() == ref["lens"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv,hd", [(4, 4, 32), (8, 2, 64), (28, 4, 128), (3, 1, 128)])
@pytest.mark.parametrize("rows,lens,pos", [
    ([1, 1, 1, 1], [0, 15, 16, 63], None),          # single tokens around a block
    ([32, 7, 0, 50], [40, 0, 9, 127], None),        # blocks, an idle sequence
    ([32], [200], [77]),                            # a diffusion block inside the sequence
    ([5, 16], [64, 100], [70, 96]),                 # behind a gap; the last, partly new block
    ([200], [0], None),                             # a prompt
])
def test_append(dtype, hq, hkv, hd, rows, lens, pos):
    g = torch.Generator().manual_seed(sum(rows) + hd + hq)
    T, starts = sum(rows), _starts(rows)
    ends = [max(L, (L if pos is None else pos[i]) + rows[i]) for i, L in enumerate(lens)]
    cache = kv8_ref.make_cache(g, ends, hkv, hd)
    for i, L in enumerate(lens):           # what lies behind lens is not a token yet
        for j, page in enumerate(cache["table"][i, :-(-ends[i] // 64)].tolist()):
            dead = max(0, -(-max(0, min(64, L - 64 * j)) // 16))
            for s in ("k_scale", "v_scale"):
                cache[s][page, :, dead:] = float("nan")
    qkv = (torch.randn(T + 2, hq + 2 * hkv, hd, generator=g) *
           torch.exp(2 * torch.randn(T + 2, 1, 1, generator=g))).to(TYPES[dtype])
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    rope = _rope(max(ends) + 1, hd)
    ref = kv8_ref.append(cache_ref := {n: t.clone() for n, t in cache.items()}, k, v, starts, lens,
                         pos, rope, q)
    d, c = _gpu(cache)
    G = qkv.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens_out = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    got = fdllm.fdllm_kv8_append(
        c, G[:, hq:hq + hkv], G[:, hq + hkv:], _i32(starts), _i32(lens),
        pos=_i32(pos) if pos else None, rope=rope.cuda(), q=G[:, :hq], max_new=max(rows),
        stored=True, lens_out=lens_out, status=status)
    _check_append(cache_ref, d, got, ref, status, lens_out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv,hd,rows,lens", [
    (36, 12, 128, [2400], [77]),      # a CTA's heads are of K, of V and of q
    (32, 32, 128, [1700], [5]),
    (40, 20, 64, [2600], [0]),
    (28, 4, 128, [500, 3, 0, 250, 100, 16, 499, 1], [3, 61, 40, 0, 1000, 64, 7, 15]),
])
def test_append_with_several_heads_a_warp(dtype, hq, hkv, hd, rows, lens):
    """Calls large enough for four heads a warp, each but the first loaded while
    the one before is worked on (float32 rows of 128 dims are not)."""
    blocks = (max(rows) + 30) // 16
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert -(-(2 * hkv + hq) // 8) * blocks * len(rows) > 8 * sms
    g = torch.Generator().manual_seed(sum(rows) + hkv)
    T, starts, ends = sum(rows), _starts(rows), [a + b for a, b in zip(lens, rows)]
    cache = kv8_ref.make_cache(g, ends, hkv, hd)
    qkv = (torch.randn(T, hq + 2 * hkv, hd, generator=g) * torch.exp(torch.randn(T, 1, 1, generator=g))).to(TYPES[dtype])
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    rope = _rope(max(ends), hd)
    ref_c = {n: t.clone() for n, t in cache.items()}
    ref = kv8_ref.append(ref_c, k, v, starts, lens, None, rope, q)
    d, c = _gpu(cache)
    G = qkv.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens_out = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    got = fdllm.fdllm_kv8_append(c, G[:, hq:hq + hkv], G[:, hq + hkv:], _i32(starts), _i32(lens), rope=rope.cuda(),
                                 q=G[:, :hq], max_new=max(rows), stored=True, lens_out=lens_out, status=status)
    _check_append(ref_c, d, got, ref, status, lens_out)


def test_append_without_rotation_hint_outputs_or_q():
    g = torch.Generator().manual_seed(3)
    rows, lens = [3, 90], [10, 31]
    cache = kv8_ref.make_cache(g, [13, 121], 2, 64)
    k, v = (torch.randn(93, 2, 64, generator=g) for _ in "kv")
    starts = _starts(rows)
    for hint in (0, 1, 1000):
        ref_c = {n: t.clone() for n, t in cache.items()}
        ref = kv8_ref.append(ref_c, k, v, starts, lens)
        d, c = _gpu(cache)
        st, lo = torch.zeros(1, dtype=torch.int32, device="cuda"), _i32([0, 0])
        got = fdllm.fdllm_kv8_append(c, k.cuda(), v.cuda(), _i32(starts), _i32(lens), max_new=hint,
                                     lens_out=lo, status=st)
        assert got == (None, None, None)
        _check_append(ref_c, d, got, ref, st, lo)


def test_append_extreme_values():
    """Zeros, infinities, NaN, the largest and the smallest numbers; a kept
    token whose block's scale grows by 2^30 and one whose new row is zero."""
    big = torch.finfo(torch.float32).max
    rows = torch.zeros(6, 1, 32)
    rows[1, 0, 3], rows[1, 0, 4], rows[1, 0, 5] = float("inf"), -float("inf"), float("nan")
    rows[1, 0, 6] = 2.0
    rows[2] = big
    rows[3] = 1e-37
    rows[4] = 1e-42
    for which, at in ((0, 0), (1, 0), (2, 0), (3, 0), (4, 0), (5, 7), (2, 7), (1, 7)):
        cache = kv8_ref.make_cache(torch.Generator().manual_seed(which), [at + 1], 1, 32)
        ref_c = {n: t.clone() for n, t in cache.items()}
        x = rows[which:which + 1]
        ref = kv8_ref.append(ref_c, x, -x, [0, 1], [at])
        d, c = _gpu(cache)
        st, lo = torch.zeros(1, dtype=torch.int32, device="cuda"), _i32([0])
        got = fdllm.fdllm_kv8_append(c, x.cuda(), (-x).cuda(), _i32([0, 1]), _i32([at]), stored=True,
                                     lens_out=lo, status=st)
        _check_append(ref_c, d, got, ref, st, lo)


def test_append_reports_what_it_cannot_store():
    g = torch.Generator().manual_seed(4)
    cache = kv8_ref.make_cache(g, [100, 100], 1, 32, extra_width=0)   # 2 pages: 128 positions
    x = torch.randn(40, 1, 32, generator=g)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    # beyond the page table: the rows that fit are stored
    ref_c = {n: t.clone() for n, t in cache.items()}
    kv8_ref.append(ref_c, x[:28], x[:28], [0, 28, 28], [100, 100])
    d, c = _gpu(cache)
    lo = _i32([0, 0])
    fdllm.fdllm_kv8_append(c, x.cuda(), x.cuda(), _i32([0, 40, 40]), _i32([100, 100]), lens_out=lo, status=st)
    assert st.item() == fdllm.KV8_BAD_RANGE and lo.tolist() == [128, 100]
    assert torch.equal(d["k"].cpu(), ref_c["k"])
    # beyond the rotation table, and a negative position: nothing is stored
    for kw in (dict(rope=_rope(100, 32).cuda()), dict(pos=_i32([-3, 0]))):
        d, c = _gpu(cache)
        st.zero_()
        fdllm.fdllm_kv8_append(c, x.cuda(), x.cuda(), _i32([0, 40, 40]), _i32([100, 100]), status=st, **kw)
        assert st.item() == fdllm.KV8_BAD_RANGE and torch.equal(d["k"].cpu(), cache["k"])
    # a bad page: its block is skipped, q is rotated all the same
    for bad in (-1, cache["k"].shape[0]):
        d, c = _gpu(cache)
        d["table"][0, 1] = bad
        st.zero_()
        q, _, _ = fdllm.fdllm_kv8_append(c, x.cuda(), x.cuda(), _i32([0, 40, 40]), _i32([60, 100]),
                                         rope=_rope(128, 32).cuda(), q=x.cuda(), status=st)
        assert st.item() == fdllm.KV8_BAD_PAGE
        want = kv8_ref.rotate(x, _rope(128, 32), torch.arange(60, 100))
        assert torch.equal(q.cpu(), want)
        other = torch.ones(cache["k"].shape[0], dtype=torch.bool)
        other[cache["table"][0, 0].long()] = False
        assert torch.equal(d["k"].cpu()[other], cache["k"][other])


def test_append_into_q_itself():
    """q_out may be q when q is dense (the C entry; the binding allocates)."""
    import ctypes
    g = torch.Generator().manual_seed(5)
    cache = kv8_ref.make_cache(g, [9], 2, 64)
    d, c = _gpu(cache)
    q = torch.randn(4, 6, 64, generator=g).to(torch.bfloat16)
    k = torch.randn(4, 2, 64, generator=g).to(torch.bfloat16)
    G, K, rope, starts, lens = q.cuda(), k.cuda(), _rope(16, 64).cuda(), _i32([0, 4]), _i32([5])
    a = fdllm.FdllmKv8AppendArgs(1, 4, 6, 0, K.data_ptr(), K.data_ptr(), G.data_ptr(), 128, 64, 128, 64,
                                 384, 64, starts.data_ptr(), lens.data_ptr(), None, rope.data_ptr(), 16, 0,
                                 None, None, G.data_ptr(), None, None)
    torch.cuda.synchronize()
    assert fdllm.load_library().fdllm_kv8_append(ctypes.byref(c.struct), ctypes.byref(a), None) == 0
    torch.cuda.synchronize()
    want = kv8_ref.rotate(q, _rope(16, 64), torch.arange(5, 9)).to(torch.bfloat16)
    assert torch.equal(G.cpu(), want)


# --------------------------------------------------------- streams, graphs, runs
def test_other_stream_and_captured_graph():
    """A captured step (append + attention, its workspace in the graph's pool)
    replayed with new inputs equals eager calls, on a side stream."""
    g = torch.Generator().manual_seed(11)
    lens = [3000, 40]
    cache = kv8_ref.make_cache(g, [3001, 41], 2, 64)
    d, c = _gpu(cache)
    qkv = torch.randn(2, 8, 64, generator=g).to(torch.bfloat16).cuda()
    starts, dl, rope = _i32([0, 1, 2]), _i32(lens), _rope(3001, 64).cuda()

    def step():
        q, _, _ = fdllm.fdllm_kv8_append(c, qkv[:, 4:6], qkv[:, 6:], starts, dl, rope=rope,
                                         q=qkv[:, :4], max_new=1, lens_out=new)
        return fdllm.fdllm_kv8_attention(c, q, starts, new, max_q=1, max_len=3008)

    new = torch.empty_like(dl)
    keep = {n: t.clone() for n, t in d.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        qkv.copy_(torch.randn(2, 8, 64, generator=g).to(torch.bfloat16))
        for n in d:
            d[n].copy_(keep[n])
        graph.replay()
        torch.cuda.synchronize()
        got, got_k = out.clone(), d["k"].clone()
        for n in d:
            d[n].copy_(keep[n])
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_k, d["k"])


def test_stream_argument():
    """Calls enqueued on another stream than torch's current one, by its
    handle: results, and workspaces, of the calls before are not handed out to
    the current stream while the other one still works with them."""
    g = torch.Generator().manual_seed(14)
    lens = [20000]
    cache = kv8_ref.make_cache(g, lens, 2, 64)
    _, c = _gpu(cache)
    q = torch.randn(8, 4, 64, generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn(8, 5000, generator=g).cuda()
    u = torch.rand(8, generator=g, dtype=torch.float64).cuda()
    starts, dl = _i32([0, 8]), _i32(lens)
    want, want_tok = fdllm.fdllm_kv8_attention(c, q, starts, dl), fdllm.fdllm_sample(logits, u)[0]
    for s in (torch.cuda.Stream(), torch.cuda.current_stream(), torch.cuda.default_stream()):
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(20):
            got = fdllm.fdllm_kv8_attention(c, q, starts, dl, stream=s.cuda_stream)
            tok, _ = fdllm.fdllm_sample(logits, u, stream=s.cuda_stream)
            torch.full((1 << 20,), 3.0, device="cuda")   # scribbles over freed memory of the current stream
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got, want) and torch.equal(tok, want_tok)


def test_integers_beyond_32_bits_are_refused():
    cache = kv8_ref.make_cache(torch.Generator().manual_seed(0), [64], 1, 64)
    _, c = _gpu(cache)
    q = torch.zeros(1, 1, 64, device="cuda")
    for kw in (dict(max_q=1 << 32), dict(max_len=-(1 << 40))):
        with pytest.raises(ValueError, match="32 bits"):
            fdllm.fdllm_kv8_attention(c, q, _i32([0, 1]), _i32([9]), **kw)
    with pytest.raises(ValueError, match="32 bits"):
        fdllm.fdllm_kv8_append(c, q, q, _i32([0, 1]), _i32([9]), max_new=1 << 32)
    with pytest.raises(ValueError, match="32 bits"):
        fdllm.fdllm_sample(q[0], torch.zeros(1, dtype=torch.float64, device="cuda"), mask_id=1 << 32)


def test_results_do_not_depend_on_timing():
    g = torch.Generator().manual_seed(12)
    lens = [4000, 129, 2000]
    cache = kv8_ref.make_cache(g, lens, 2, 128)
    _, c = _gpu(cache)
    q = torch.randn(3 * 20, 8, 128, generator=g).to(torch.float16).cuda()
    runs = [fdllm.fdllm_kv8_attention(c, q, _i32([0, 20, 40, 60]), _i32(lens)) for _ in range(5)]
    assert all(torch.equal(r, runs[0]) for r in runs)


def test_decode_loop_on_the_cache():
    """Prompt, then diffusion blocks rewritten in place and single tokens: the
    cache's tokens, and what attention reads, stay those of the plain loop."""
    g = torch.Generator().manual_seed(13)
    hq, hkv, hd = 8, 2, 64
    cache = kv8_ref.make_cache(g, [300, 300], hkv, hd)
    for s in ("k_scale", "v_scale"):
        cache[s].fill_(float("nan"))
    ref_c = {n: t.clone() for n, t in cache.items()}
    d, c = _gpu(cache)
    rope = _rope(300, hd)
    lens = [0, 0]
    #      rows           positions
    plan = [([70, 101], [0, 0]), ([32, 32], [70, 101]), ([32, 32], [70, 101]), ([32, 0], [70, 133]),
            ([1, 1], [102, 133]), ([1, 1], [103, 134]), ([32, 32], [104, 135])]
    for rows, pos in plan:
        starts = _starts(rows)
        qkv = torch.randn(sum(rows), hq + 2 * hkv, hd, generator=g).to(torch.bfloat16)
        ref = kv8_ref.append(ref_c, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], starts, lens, pos, rope, qkv[:, :hq])
        G, new = qkv.cuda(), _i32([0, 0])
        q, _, _ = fdllm.fdllm_kv8_append(c, G[:, hq:hq + hkv], G[:, hq + hkv:], _i32(starts), _i32(lens),
                                         pos=_i32(pos), rope=rope.cuda(), q=G[:, :hq], lens_out=new)
        lens = ref["lens"]
        assert new.tolist() == lens
        assert torch.equal(d["k"].cpu(), ref_c["k"]) and torch.equal(d["v"].cpu(), ref_c["v"])
        got = fdllm.fdllm_kv8_attention(c, q, _i32(starts), new)
        _check_attention(ref_c, ref["q"], starts, lens, hd ** -0.5, got)


@pytest.mark.parametrize("n,rows,hq,hkv", [(64, 1, 28, 4), (16, 32, 32, 32), (16, 32, 28, 4), (1, 70, 8, 2), (7, 3, 8, 8)])
def test_a_batch_is_laid_out_alike_with_and_without_hints(n, rows, hq, hkv):
    """n sequences of as many rows: without max_q the rows of one are taken to be
    n_tokens / n_seqs, so the same kernel, grid and workspace, and the same bits."""
    g = torch.Generator().manual_seed(21)
    lens = [int(x) for x in torch.randint(1, 400, (n,), generator=g)]
    cache = kv8_ref.make_cache(g, lens, hkv, 128)
    _, c = _gpu(cache)
    q = torch.randn(n * rows, hq, 128, generator=g).to(torch.bfloat16)
    a, b = (fdllm.fdllm_kv8_attention_workspace(c, n * rows, hq, q.dtype, m, 64 * c.max_pages) for m in (0, rows))
    assert a == b
    starts, dl = _i32([rows * i for i in range(n + 1)]), _i32(lens)
    got, want = (fdllm.fdllm_kv8_attention(c, q.cuda(), starts, dl, max_q=m) for m in (0, rows))
    assert torch.equal(got, want)


@pytest.mark.parametrize("hq,hkv,rows", [(32, 32, 32), (16, 16, 64), (28, 4, 16), (28, 4, 32)])
def test_many_runs_repeat_to_the_bit(hq, hkv, rows):
    """Ragged batches whose CTAs start and end several runs each: every call
    gives the same bits."""
    g = torch.Generator().manual_seed(15)
    lens = [int(x) for x in torch.randint(1, 1300, (16,), generator=g)]
    cache = kv8_ref.make_cache(g, lens, hkv, 128)
    _, c = _gpu(cache)
    q = torch.randn(16 * rows, hq, 128, generator=g).to(torch.float16).cuda()
    starts, dl = _i32([rows * i for i in range(17)]), _i32(lens)
    first = fdllm.fdllm_kv8_attention(c, q, starts, dl, max_q=rows, max_len=1300)
    for _ in range(40):
        assert torch.equal(fdllm.fdllm_kv8_attention(c, q, starts, dl, max_q=rows, max_len=1300), first)


@pytest.mark.parametrize("hq,hkv,hd,rows", [(28, 4, 128, 16), (28, 4, 128, 32), (8, 2, 64, 40), (16, 4, 64, 21)])
def test_grouped_blocks_stay_the_same_over_many_calls(hq, hkv, hd, rows):
    """Runs of 112, 224, 160 and 84 rows a K/V head: 1500 calls give the bits of the
    first, alone, with a matrix product on another stream beside them, and with
    the same call on another stream."""
    g = torch.Generator().manual_seed(17)
    lens = [int(x) for x in torch.randint(1, 1300, (16,), generator=g)]
    cache = kv8_ref.make_cache(g, lens, hkv, hd)
    _, c = _gpu(cache)
    q = torch.randn(16 * rows, hq, hd, generator=g).to(torch.float16)
    Q, starts, dl = q.cuda(), _i32([rows * i for i in range(17)]), _i32(lens)

    def call():
        return fdllm.fdllm_kv8_attention(c, Q, starts, dl, max_q=rows, max_len=1300)

    first = call()
    _check_attention(cache, q, starts.tolist(), lens, hd ** -0.5, first)
    bad = torch.zeros(2, dtype=torch.int64, device="cuda")
    a = torch.randn(2048, 2048, device="cuda").to(torch.bfloat16)
    s = torch.cuda.Stream()
    for beside in (None, "product", "call"):
        s.wait_stream(torch.cuda.current_stream())
        for i in range(500):
            if beside is not None:
                with torch.cuda.stream(s):
                    if beside == "product":
                        a @ a
                    else:
                        bad[1] += (call() != first).any()
            bad[0] += (call() != first).any()
        torch.cuda.synchronize()
    assert bad.tolist() == [0, 0]
