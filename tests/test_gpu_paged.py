"""The paged-cache operators on the GPU against 64-bit references."""
import math

import pytest
import torch

import shared_kv_cache_gb300 as gqa

from paged_cases import (Case, assert_close, caches, ref_attention, ref_kept, ref_rows, ref_weights, rotate_fp32,
                         same_bits, visible)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gqa.load_library()


def ok():
    st = gqa.gqa_check_device_status(torch.cuda.current_stream())
    assert st == gqa.GQA_OK, gqa.gqa_status_string(st)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def rows_of(c, positions=None):
    """(row of the token arrays, sequence, slot) of every new token."""
    return [(int(c.cu[b]) + i, b, c.past[b] + i) for b in range(c.B) for i in range(c.new[b])]


def check_append(c, norm=True, rotary=True, interleaved=0, packed=False, positions=None, in_place=False):
    g = torch.Generator().manual_seed(99)
    D, t = c.D, c.t
    d = c.cuda()
    qw = kw = cos = sin = None
    if norm:
        qw, kw = (1 + 0.3 * torch.randn(D, generator=g)).to(t), (1 + 0.3 * torch.randn(D, generator=g)).to(t)
    rows = max(c.total, 1 if positions is None else int(positions.max()) + 1)
    if rotary:
        cos, sin = caches(rows, D, c.dtype)
    up = lambda x: None if x is None else x.cuda()  # noqa: E731
    n_rows = c.query.shape[0]
    sentinel = torch.full((n_rows, c.H * D), 7.0, dtype=t, device="cuda")
    kp0, vp0 = d["k_pages"].clone(), d["v_pages"].clone()
    if packed:
        q = torch.cat([d["query"], d["key"], d["value"]], 1).contiguous()
        args = (q, None, None)
    else:
        args = (d["query"], d["key"], d["value"])
    out = d["query"] if in_place else sentinel
    got = gqa.paged_append(*args, d["k_pages"], d["v_pages"], d["table"], d["cu"], d["seqlens"], c.total, up(qw),
                           up(kw), 1e-5, up(cos), up(sin), up(positions), query_out=out,
                           rotary_interleaved=interleaved)
    ok()
    assert got.data_ptr() == out.data_ptr()
    where = rows_of(c)
    r = torch.tensor([x[0] for x in where])
    pos = torch.tensor([x[2] for x in where]) if positions is None else positions[r].long()
    cr, sr = (cos[pos], sin[pos]) if rotary else (None, None)
    ref_q, tol_q = ref_rows(c.query[r].view(len(r), c.H, D), qw, 1e-5, cr, sr, interleaved, c.dtype)
    ref_k, tol_k = ref_rows(c.key[r].view(len(r), c.Hkv, D), kw, 1e-5, cr, sr, interleaved, c.dtype)
    got = got.cpu()
    assert_close(got[r].view(len(r), c.H, D), ref_q, tol_q, "queries")
    rest = torch.ones(n_rows, dtype=torch.bool)
    rest[r] = False
    assert same_bits(got[rest], (c.query if in_place else sentinel.cpu())[rest]), "rows that belong to nobody"
    pg = torch.stack([c.table[b, s // c.page] for _, b, s in where]).long()
    off = torch.tensor([s % c.page for _, _, s in where])
    kp, vp = d["k_pages"].cpu(), d["v_pages"].cpu()
    assert_close(kp[pg, :, off], ref_k, tol_k, "keys")
    assert same_bits(vp[pg, :, off], c.value[r].view(len(r), c.Hkv, D)), "values"
    kp0, vp0 = kp0.cpu(), vp0.cpu()
    kp[pg, :, off] = 0
    vp[pg, :, off] = 0
    kp0[pg, :, off] = 0
    vp0[pg, :, off] = 0
    assert same_bits(kp, kp0) and same_bits(vp, vp0), "other slots"
    if rotary and not norm:
        want = rotate_fp32(c.query[r].view(len(r), c.H, D), cr, sr, interleaved).to(t)
        assert same_bits(got[r].view(len(r), c.H, D), want), "rotation without norm is bit exact"


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [8, 24, 64, 72, 80, 128, 200, 248, 256])
@pytest.mark.parametrize("interleaved", [0, 1])
def test_append_head_sizes(dtype, D, interleaved):
    c = Case(dtype, H=6, Hkv=2, D=D, past=(3, 0, 17, 30), new=(5, 1, 0, 20), seed=D, fill_new=False)
    check_append(c, interleaved=interleaved)
    check_append(c, norm=False, interleaved=interleaved)


@pytest.mark.parametrize("page", [8, 16, 256, 1024])
@pytest.mark.parametrize("packed", [False, True])
def test_append_pages_and_packing(page, packed):
    c = Case("bf16", H=10, Hkv=2, page=page, past=(1030, 7, 0), new=(9, 33, 2), seed=page, fill_new=False)
    check_append(c, packed=packed)
    check_append(c, packed=packed, rotary=False)
    check_append(c, packed=packed, rotary=False, norm=False)


def test_append_many_sequences_and_positions():
    """More sequences than a warp has lanes, some without new tokens; rotary
    positions apart from the slots; the queries in place."""
    n = 1100
    new = [(b * 7) % 3 for b in range(n)]
    c = Case("fp16", H=4, Hkv=4, D=64, page=8, past=[b % 11 for b in range(n)], new=new, seed=3, fill_new=False)
    pos = torch.randint(0, 5000, (c.query.shape[0],), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    check_append(c, positions=pos)
    check_append(c, in_place=True)


def test_append_long_prompt():
    check_append(Case("bf16", H=8, Hkv=2, page=64, past=(0, 5), new=(700, 411), seed=5, fill_new=False))


def test_append_matches_the_shared_buffers_append():
    """The keys that gqa.forward writes into its shared buffer, bit for bit."""
    from gqa_cases import custom, run_cuda
    inp = custom(dtype="bf16", B=2, S=6, H=8, Hkv=2, D=128, M=64, past=(3, 20), seed=11)
    st, dst, _, kb, _ = run_cuda(inp)
    assert st == gqa.GQA_OK and dst == gqa.GQA_OK
    kp = torch.zeros(8, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    cu = torch.tensor([0, 6, 12], dtype=torch.int32, device="cuda")
    gqa.paged_append(inp["query"].cuda().flatten(0, 1), inp["key"].cuda().flatten(0, 1),
                     inp["value"].cuda().flatten(0, 1), kp, vp, table, cu, inp["seqlens_k"].cuda(), 26,
                     cos_cache=inp["cos"].cuda(), sin_cache=inp["sin"].cuda())
    ok()
    for b, p in enumerate((3, 20)):
        rows = kp.view(2, 4, 2, 16, 128)[b].transpose(0, 1).reshape(2, 64, 128)
        assert same_bits(rows[:, p:p + 6], kb[b, :, p:p + 6])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def run_attention(c, d=None, workspace=None, with_lse=True, **over):
    d = c.cuda() if d is None else d
    out = torch.full_like(d["query"], 7.0)
    lse = torch.full((d["query"].shape[0], c.H), 7.0, device="cuda") if with_lse else None
    gqa.paged_attention(d["query"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["seqlens"],
                        over.get("max_new", c.max_new), over.get("total", c.total), c.scale, c.window, output=out,
                        lse=lse, workspace=workspace)
    return out, lse


def check_attention(c, **over):
    out, lse = run_attention(c, **over)
    ok()
    ro, rl, to, tl = ref_attention(c)
    n = c.tokens
    assert_close(out[:n].view(n, c.H, c.D), ro[:n], to[:n], "output")
    assert_close(lse[:n], rl[:n], tl[:n], "lse")
    assert (out[n:] == 7).all() and (lse[n:] == 7).all(), "rows that belong to nobody"


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [8, 64, 80, 128, 256])
def test_attention_head_sizes(dtype, D):
    check_attention(Case(dtype, H=6, Hkv=2, D=D, past=(3, 0, 17, 130), new=(5, 1, 0, 20), seed=D))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_attention_pages(D, page, new):
    """Lengths around the edges of pages and tiles."""
    past = (0, 1, 15, 16, 62, 63, 64, 65, 127, 128, 129, 255, 256, 700)
    check_attention(Case("bf16", H=8, Hkv=2, D=D, page=page, past=past, new=[new] * len(past), seed=page))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 16, 24, 71])
@pytest.mark.parametrize("new", [1, 2, 9])
def test_attention_groups(dtype, group, new):
    check_attention(Case(dtype, H=2 * group, Hkv=2, D=128, page=32, past=(0, 77, 300), new=(new, new, 1),
                         seed=group))


def test_attention_group_beyond_a_tile():
    check_attention(Case("bf16", H=130, Hkv=1, D=64, page=32, past=(0, 77), new=(2, 1), seed=4))


@pytest.mark.parametrize("D", [64, 128, 40])
@pytest.mark.parametrize("new", [1, 6, 150])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 5000])
def test_attention_window(D, new, window):
    """Pages wholly before the window hold nonsense in the table."""
    c = Case("fp16", H=4, Hkv=2, D=D, page=16, past=(0, 10, 64, 500, 1000), new=[new] * 5, window=window, seed=window)
    for b in range(c.B):
        first = max(0, c.past[b] + 1 - window)
        c.table[b, :first // c.page] = -5
        if first % c.page:  # rows before the window in its first page
            pg = int(c.table[b, first // c.page])
            c.v_pages[pg, :, :first % c.page] = float("inf")
            c.k_pages[pg, :, :first % c.page] = float("nan")
    out, lse = run_attention(c)
    ok()
    # the reference gathers every slot: give it harmless pages there
    r = Case("fp16", H=4, Hkv=2, D=D, page=16, past=c.past, new=c.new, window=window, seed=window)
    ro, rl, to, tl = ref_attention(r)
    n = c.tokens
    assert_close(out[:n].view(n, c.H, c.D), ro[:n], to[:n], "output")
    assert_close(lse[:n], rl[:n], tl[:n], "lse")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_mixed_batch(dtype):
    """A long prompt, chunks on long pasts, single tokens, idle sequences."""
    check_attention(Case(dtype, H=8, Hkv=2, D=128, page=16, past=(0, 1500, 2000, 0, 9, 777, 0),
                         new=(400, 130, 1, 0, 1, 33, 1), seed=21))


def test_attention_many_items():
    """Whole items by ticket (many blocks, none large), and many cut ones."""
    check_attention(Case("fp16", H=16, Hkv=8, D=64, page=32, past=(0, 100, 0, 300, 20, 0), seed=31,
                         new=(2000, 1500, 1, 700, 1800, 900)))
    check_attention(Case("bf16", H=16, Hkv=16, D=128, page=16, past=(3000, 2000), new=(200, 300), seed=32))
    check_attention(Case("bf16", H=8, Hkv=1, D=128, page=128, past=(30000,), new=(40,), seed=33))


@pytest.mark.parametrize("D", [64, 128])
def test_attention_large_scores(D):
    """One-hot softmax rows and scores of several hundred."""
    check_attention(Case("bf16", H=4, Hkv=1, D=D, page=32, past=(200, 30), new=(70, 1), qk=6.0, seed=2))
    check_attention(Case("fp16", H=4, Hkv=1, D=D, page=32, past=(900, 3), new=(2, 1), qk=5.0, scale=0.5, seed=3))


def test_attention_long_single_rows():
    check_attention(Case("bf16", H=4, Hkv=1, D=128, page=64, past=(20000, 1, 9000), new=(1, 1, 1), seed=8))
    check_attention(Case("fp16", H=2, Hkv=1, D=64, page=16, past=(12000,), new=(3,), seed=9))


def test_attention_many_sequences():
    n = 300
    check_attention(Case("bf16", H=4, Hkv=1, D=64, page=8, past=[(b * 13) % 90 for b in range(n)],
                         new=[b % 3 for b in range(n)], seed=10))
    check_attention(Case("bf16", H=4, Hkv=1, D=128, page=16, past=[(b * 13) % 190 for b in range(n)],
                         new=[30 if b % 50 == 0 else b % 2 for b in range(n)], seed=10))


def test_attention_block_counts_beyond_the_class_list():
    """Many sequences and a large bound on their new tokens: the partition adds a
    sequence's blocks up instead of listing them."""
    n = 300
    check_attention(Case("bf16", H=4, Hkv=1, D=64, page=8, past=[(b * 13) % 90 for b in range(n)],
                         new=[400 if b == 77 else b % 2 for b in range(n)], seed=10))


@pytest.mark.parametrize("max_new", [1, 200])
def test_nothing_new(max_new):
    """Sequences without new tokens: nothing is written."""
    c = Case("bf16", H=8, Hkv=2, D=128, page=16, past=(30, 0, 7), new=(0, 0, 0), seed=12)
    out, lse = run_attention(c, max_new=max_new, total=60)
    d = c.cuda()
    w0 = d["weights"].clone()
    gqa.paged_key_weights(d["query"], lse, d["k_pages"], d["weights"], d["table"], d["cu"], d["seqlens"], max_new, 60)
    k0 = d["k_pages"].clone()
    q = torch.full_like(d["query"], 7.0)
    gqa.paged_append(d["query"], d["key"], d["value"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["seqlens"],
                     60, query_out=q)
    ok()
    assert (out == 7).all() and (lse == 7).all() and (q == 7).all()
    assert same_bits(d["weights"], w0) and same_bits(d["k_pages"], k0)


def test_attention_same_bits_every_time():
    """Cut items are merged by whichever piece ends last: the sum's order does
    not depend on it."""
    for c in (Case("bf16", H=8, Hkv=1, D=128, page=128, past=(30000, 100), new=(40, 9), seed=33),
              Case("fp16", H=8, Hkv=2, D=64, page=16, past=(9000, 50), new=(2, 3), seed=34)):
        d = c.cuda()
        runs = [run_attention(c, d) for _ in range(6)]
        ok()
        for out, lse in runs[1:]:
            assert same_bits(out, runs[0][0]) and same_bits(lse, runs[0][1])


def test_rows_beyond_4_gib():
    """Pages whose rows lie beyond 2^32 bytes of the pools."""
    page, hkv, D = 64, 2, 128
    n_pages = (5 << 30) // (page * hkv * D * 2)
    free, _ = torch.cuda.mem_get_info()
    if free < (14 << 30):
        pytest.skip("needs 14 GiB")
    kp = torch.zeros(n_pages, hkv, page, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    wt = torch.zeros(n_pages, hkv, page, device="cuda")
    for new in (1, 50):
        c = Case("bf16", H=8, Hkv=hkv, D=D, page=page, past=(200, 77), new=(new, new), seed=1)
        used = c.num_pages
        d = c.cuda()
        kp[n_pages - used:] = d["k_pages"]
        vp[n_pages - used:] = d["v_pages"]
        wt[n_pages - used:] = d["weights"]
        big = torch.where((c.table >= 0) & (c.table < used), c.table + (n_pages - used), c.table)
        out, lse = torch.empty_like(d["query"]), torch.empty(d["query"].shape[0], c.H, device="cuda")
        args = (big.cuda(), d["cu"], d["seqlens"])
        gqa.paged_attention(d["query"], kp, vp, *args, c.max_new, c.total, output=out, lse=lse)
        gqa.paged_key_weights(d["query"], lse, kp, wt, *args, c.max_new, c.total)
        ok()
        ro, rl, to, tl = ref_attention(c)
        n = c.tokens
        assert_close(out[:n].view(n, c.H, c.D), ro[:n], to[:n], "output")
        rw, tw, written = ref_weights(c, lse.cpu())
        assert_close(wt[n_pages - used:].cpu()[written], rw[written], tw[written], "weights")
        kept, _ = gqa.paged_evict(kp, vp, wt, big.cuda(), d["seqlens"], c.total, 50, 10)
        ok()
        w = wt  # in place: the first kept row of sequence 0, head 0 holds its old slot's key
        src = c.gather(c.k_pages, 0, c.past[0])[0, int(kept[0, 0, 0])]
        assert same_bits(kp[int(big[0, 0]), 0, 0], src)
        g = torch.Generator().manual_seed(2)
        key = torch.randn(c.tokens, hkv * D, generator=g).to(torch.bfloat16).cuda()
        gqa.paged_append(d["query"][:n], key, key, kp, vp, *args, c.total)
        ok()
        s = c.past[0]
        assert same_bits(kp[int(big[0, s // page]), :, s % page], key[0].view(hkv, D))


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp16"), (40, "fp16")])
@pytest.mark.parametrize("past,new,window", [((40, 700), (3, 2), 0), ((40, 700), (3, 2), 2), ((500, 3), (70, 150), 0),
                                             ((500, 3), (70, 150), 50), ((9000,), (40,), 0), ((9000,), (3,), 0),
                                             ((9000,), (60,), 20)])
def test_attention_values_that_are_not_finite(D, dtype, past, new, window):
    """Infinities and NaN in value rows (and a key row) of some new tokens, and
    of tokens that leave the window: they reach the tokens that see them, in
    the dimensions that have them, and no others."""
    c = Case(dtype, H=4, Hkv=1, D=D, page=16, past=past, new=new, window=window, seed=7)
    g = torch.Generator().manual_seed(3)
    clean_k, clean_v = c.k_pages.clone(), c.v_pages.clone()
    odd = torch.zeros(c.k_pages.shape, dtype=torch.bool)          # value elements
    nan_keys = torch.zeros(c.k_pages.shape[:3], dtype=torch.bool)
    for b in range(c.B):
        slots = {past[b] + new[b] - 1, past[b] + new[b] // 2, past[b] + 1}
        if window:
            slots |= {max(0, past[b] + 1 - window), max(0, past[b] + 2 - window)}
        for j in slots:
            pg, off = int(c.table[b, j // 16]), j % 16
            dims = torch.randperm(D, generator=g)[:5]
            c.v_pages[pg, 0, off, dims] = torch.tensor([math.inf, -math.inf, math.nan, math.inf, math.nan]).to(c.t)
            odd[pg, 0, off, dims] = True
        j = past[b] + new[b] - 1
        c.k_pages[int(c.table[b, j // 16]), 0, j % 16, 2] = math.nan
        nan_keys[int(c.table[b, j // 16]), 0, j % 16] = True
    out, lse = run_attention(c)
    ok()
    zero_v = torch.where(odd, torch.zeros((), dtype=c.t), clean_v)
    ro, rl, to, tl = ref_attention(c, clean_k, zero_v)
    for b in range(c.B):
        seen = visible(c, b).double()
        L = past[b] + new[b]
        hit_v = (seen @ c.gather(odd, b, L)[0].double()) > 0             # [new, D]
        hit_k = (seen @ c.gather(nan_keys, b, L)[0].double()) > 0        # [new]
        r = slice(int(c.cu[b]), int(c.cu[b + 1]))
        got = out[r].cpu().view(new[b], c.H, D).double()
        bad = (hit_v | hit_k[:, None])[:, None].expand_as(got)
        assert not torch.isfinite(got[bad]).any()
        assert_close(torch.where(bad, torch.zeros(()), got), torch.where(bad, torch.zeros(()), ro[r]), to[r], "output")
        ll = lse[r].cpu().double()
        assert torch.isnan(ll[hit_k]).all()
        assert_close(ll[~hit_k], rl[r][~hit_k], tl[r][~hit_k], "lse")


def test_attention_bounds_may_be_loose():
    c = Case("bf16", H=8, Hkv=2, D=128, page=16, past=(30, 200), new=(1, 2), seed=12)
    c.table = torch.cat([c.table, torch.full((2, 200), -1, dtype=torch.int32)], 1)
    check_attention(c, max_new=500, total=3000)


def test_attention_without_lse_and_with_one_workspace():
    """One workspace for calls of different shapes; equal calls give equal bits
    without partials' order mattering."""
    ws = gqa.Workspace()
    a = Case("bf16", H=32, Hkv=8, D=128, page=16, past=(300, 900, 5), new=(1, 1, 1), seed=13)
    b = Case("fp16", H=8, Hkv=2, D=64, page=32, past=(100, 2000), new=(64, 7), seed=14)
    for c in (a, b, a, b):
        out, _ = run_attention(c, workspace=ws, with_lse=False)
        ok()
        ro, _, to, _ = ref_attention(c)
        assert_close(out[:c.tokens].view(c.tokens, c.H, c.D), ro[:c.tokens], to[:c.tokens], "output")


# ---------------------------------------------------------------------------
# key weights
# ---------------------------------------------------------------------------
def check_weights(c, in_place=False):
    _, lse64, _, _ = ref_attention(c)
    lse = lse64.float()
    d = c.cuda()
    before = d["weights"].clone() if in_place else torch.full_like(d["weights"], 3.0)
    w = d["weights"] if in_place else before.clone()
    got = gqa.paged_key_weights(d["query"], lse.cuda(), d["k_pages"], w, d["table"], d["cu"], d["seqlens"], c.max_new,
                                c.total, c.scale, c.window, weights_in=None if in_place else d["weights"])
    ok()
    assert got.data_ptr() == w.data_ptr()
    ref, tol, written = ref_weights(c, lse)
    got = got.cpu()
    assert_close(got[written], ref[written], tol[written], "weights")
    assert same_bits(got[~written], before.cpu()[~written]), "slots out of reach"


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [8, 64, 80, 128, 256])
@pytest.mark.parametrize("in_place", [False, True])
def test_weights_head_sizes(dtype, D, in_place):
    check_weights(Case(dtype, H=6, Hkv=2, D=D, past=(3, 0, 17, 130), new=(5, 1, 0, 20), seed=D), in_place)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 64, 128, 512])
@pytest.mark.parametrize("new", [1, 4, 150])
def test_weights_pages(D, page, new):
    past = (0, 1, 15, 64, 127, 128, 129, 700)
    check_weights(Case("bf16", H=8, Hkv=2, D=D, page=page, past=past, new=[new] * len(past), seed=page))


@pytest.mark.parametrize("group", [1, 3, 7, 16, 71])
@pytest.mark.parametrize("new", [1, 9])
def test_weights_groups(group, new):
    check_weights(Case("fp16", H=2 * group, Hkv=2, D=128, page=32, past=(0, 77, 300), new=(new, new, 1), seed=group))


@pytest.mark.parametrize("new", [1, 6, 150])
@pytest.mark.parametrize("window", [1, 63, 64, 200])
def test_weights_window(new, window):
    check_weights(Case("bf16", H=4, Hkv=2, D=128, page=16, past=(0, 10, 64, 500), new=[new] * 4, window=window,
                       seed=window))


def test_weights_long_and_large():
    check_weights(Case("bf16", H=4, Hkv=1, D=128, page=64, past=(9000, 1), new=(2, 1), seed=8))
    check_weights(Case("bf16", H=4, Hkv=1, D=64, page=32, past=(200, 30), new=(70, 1), qk=4.0, seed=2))
    check_weights(Case("fp16", H=8, Hkv=1, D=64, page=32, past=(0, 40), new=(500, 300), seed=2))


def test_weights_many_items():
    """More items than a CTA's descriptor ring has places, several blocks each."""
    check_weights(Case("fp16", H=8, Hkv=8, D=64, page=16, past=(1000, 3000, 2500, 7), new=(300, 260, 130, 290), seed=3))
    check_weights(Case("bf16", H=32, Hkv=16, D=128, page=64, past=(900, 5000, 2500), new=(130, 70, 200), seed=3))
    check_weights(Case("bf16", H=16, Hkv=16, D=128, page=64, past=(9000, 5000, 7500), new=(1, 1, 1), seed=3))


def test_weights_are_the_same_every_time():
    c = Case("bf16", H=8, Hkv=2, D=128, page=16, past=(700, 64), new=(90, 5), seed=4)
    d = c.cuda()
    _, lse = run_attention(c, d)
    got = [gqa.paged_key_weights(d["query"], lse, d["k_pages"], torch.zeros_like(d["weights"]), d["table"], d["cu"],
                                 d["seqlens"], c.max_new, c.total, weights_in=d["weights"]) for _ in range(3)]
    ok()
    assert same_bits(got[0], got[1]) and same_bits(got[0], got[2])


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def check_evict(c, budget, recent, in_place, weights=None, total=None):
    d = c.cuda()
    if weights is not None:
        c.weights = weights
        d["weights"] = weights.cuda()
    dst = None
    per = -(-budget // c.page)
    table2 = c.table
    if not in_place:
        # pages of its own for every sequence, behind the pool's
        extra = c.B * per
        grow = lambda x: torch.cat([x, torch.full((extra,) + x.shape[1:], float("nan"), dtype=x.dtype)])  # noqa: E731
        for n in ("k_pages", "v_pages", "weights"):
            setattr(c, n, grow(getattr(c, n)))
            d[n] = getattr(c, n).cuda()
        order = torch.randperm(extra, generator=torch.Generator().manual_seed(1)).to(torch.int32) + c.num_pages
        table2 = order.view(c.B, per)
        dst = table2.cuda()
        c.num_pages += extra
    kept, left = gqa.paged_evict(d["k_pages"], d["v_pages"], d["weights"], d["table"], d["seqlens"],
                                 c.total if total is None else total, budget, recent, dst_block_table=dst)
    ok()
    kept, left = kept.cpu(), left.cpu()
    want = {n: getattr(c, n).clone() for n in ("k_pages", "v_pages", "weights")}
    for b in range(c.B):
        n = c.past[b]
        assert left[b] == min(n, budget)
        w = c.gather(c.weights, b, n)
        for h in range(c.Hkv):
            keep = ref_kept(w[h].tolist(), recent, budget)
            assert kept[b, h].tolist() == keep + [-1] * (budget - len(keep)), (b, h)
            if not keep:
                continue
            k = torch.tensor(keep)
            j = torch.arange(len(keep))
            for x in want:
                src = getattr(c, x)
                want[x][table2[b, j // c.page].long(), h, j % c.page] = src[c.table[b, k // c.page].long(), h, k % c.page]
    for x in want:
        assert same_bits(d[x], want[x]), x


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (16, 0), (40, 8), (40, 40), (129, 64), (600, 100), (5000, 7)])
def test_evict(in_place, budget, recent):
    check_evict(Case("bf16", Hkv=3, H=3, D=128, page=16, past=(0, 1, 16, 40, 41, 130, 700, 1333), new=[0] * 8,
                     seed=budget), budget, recent, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D,page,dtype", [(8, 8, "fp16"), (64, 64, "bf16"), (80, 32, "fp16"), (256, 1024, "bf16")])
def test_evict_layouts(in_place, D, page, dtype):
    check_evict(Case(dtype, Hkv=2, H=2, D=D, page=page, past=(300, 77, 2500), new=[0] * 3, seed=D), 200, 30, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_special_weights(in_place):
    """Ties (the lower slot), signed zeros, infinities, NaN, negative values,
    subnormals."""
    c = Case("fp16", Hkv=4, H=4, D=16, page=16, past=(500, 300, 1200), new=[0] * 3, seed=1)
    pool = torch.tensor([0.0, -0.0, 1.0, 1.0, -1.0, math.inf, -math.inf, math.nan, 1e-40, -1e-40, 3.5, 2.0 ** -126])
    pick = torch.randint(0, len(pool), c.weights.shape, generator=torch.Generator().manual_seed(5))
    for budget, recent in ((100, 10), (250, 0), (299, 299)):
        cc = Case("fp16", Hkv=4, H=4, D=16, page=16, past=(500, 300, 1200), new=[0] * 3, seed=1)
        check_evict(cc, budget, recent, in_place, weights=pool[pick].clone())
    same = torch.full_like(c.weights, 0.25)
    check_evict(c, 123, 20, in_place, weights=same)


def test_evict_long():
    c = Case("bf16", Hkv=2, H=2, D=64, page=64, past=(33000, 70001, 10), new=[0] * 3, seed=6)
    check_evict(c, 4096, 256, True)
    check_evict(Case("bf16", Hkv=2, H=2, D=64, page=64, past=(33000, 70001, 10), new=[0] * 3, seed=6), 9000, 0, False)


# ---------------------------------------------------------------------------
# the run of them, as a server uses them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp16"), (40, "fp16")])
def test_serving_run(D, dtype):
    """Prompts in chunks, decode steps, an eviction in place, more decode with
    positions apart from slots: outputs against a dense float64 model of the
    same cached rows, kept tokens against the weights the kernels summed."""
    B, H, Hkv, page, cols, budget, recent = 3, 8, 2, 16, 20, 96, 24
    G = H // Hkv
    g = torch.Generator().manual_seed(7)
    base = Case(dtype, H=H, Hkv=Hkv, D=D, page=page, past=(0,) * B, new=(0,) * B, seed=1)
    t = base.t
    n_pages = B * cols
    kp = torch.full((n_pages, Hkv, page, D), float("nan"), dtype=t, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    wt = torch.full((n_pages, Hkv, page), float("nan"), device="cuda")
    table = torch.randperm(n_pages, generator=g).to(torch.int32).view(B, cols)
    qw, kw = (1 + 0.2 * torch.randn(D, generator=g)).to(t), (1 + 0.2 * torch.randn(D, generator=g)).to(t)
    cos, sin = caches(400, D, dtype)
    lens, seen = [0] * B, [0] * B
    ws = gqa.Workspace()
    steps = [(60, 5, 17), (50, 40, 0), (1, 1, 1), (30, 100, 70), (1, 1, 1), "evict", (1, 1, 1), (9, 3, 0), (1, 1, 1)]
    for step in steps:
        if step == "evict":
            before = {n: x.cpu().clone() for n, x in (("k", kp), ("v", vp), ("w", wt))}
            sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
            kept, left = gqa.paged_evict(kp, vp, wt, table.cuda(), sl, max(lens), budget, recent)
            ok()
            for b in range(B):
                j = torch.arange(lens[b])
                w = before["w"][table[b, j // page].long(), :, j % page].T
                for h in range(Hkv):
                    keep = ref_kept(w[h].tolist(), recent, budget)
                    assert kept[b, h].tolist() == keep + [-1] * (budget - len(keep))
            lens = left.cpu().tolist()
            continue
        c = Case(dtype, H=H, Hkv=Hkv, D=D, page=page, past=lens, new=step, seed=100 + sum(step))
        c.table = table
        pos = torch.zeros(c.query.shape[0], dtype=torch.int32)
        for b in range(B):
            pos[int(c.cu[b]):int(c.cu[b + 1])] = torch.arange(seen[b], seen[b] + step[b], dtype=torch.int32)
        d = {n: getattr(c, n).cuda() for n in ("query", "key", "value", "table", "cu", "seqlens")}
        tail = (d["table"], d["cu"], d["seqlens"])
        q = gqa.paged_append(d["query"], d["key"], d["value"], kp, vp, *tail, c.total, qw.cuda(), kw.cuda(), 1e-6,
                             cos.cuda(), sin.cuda(), pos.cuda())
        lse = torch.empty(q.shape[0], H, device="cuda")
        out = gqa.paged_attention(q, kp, vp, *tail, c.max_new, c.total, lse=lse, workspace=ws)
        old = wt.cpu().clone()
        gqa.paged_key_weights(q, lse, kp, wt, *tail, c.max_new, c.total, workspace=ws)
        ok()
        # the queries as the kernel left them; the cached rows as they are
        n = c.tokens
        r = torch.arange(n)
        ref_q, tol_q = ref_rows(c.query[:n].view(n, H, D), qw, 1e-6, cos[pos[r].long()], sin[pos[r].long()], 0, dtype)
        assert_close(q[:n].view(n, H, D), ref_q, tol_q, "queries")
        qc = q.cpu()
        ro, rl, to, tl = ref_attention(c, kp.cpu(), vp.cpu(), qc)
        assert_close(out[:n].view(n, H, D), ro[:n], to[:n], "output")
        assert_close(lse[:n], rl[:n], tl[:n], "lse")
        rw, tw, written = ref_weights(c, lse.cpu(), old, kp.cpu(), qc)
        assert_close(wt.cpu()[written], rw[written], tw[written], "weights")
        lens = [a + b for a, b in zip(lens, step)]
        seen = [a + b for a, b in zip(seen, step)]
        # each (token, head) has handed out a weight of one (before any eviction)
        if max(lens) == max(seen):
            total = sum(wt.cpu()[table[b, torch.arange(lens[b]) // page].long(), :, torch.arange(lens[b]) % page].sum()
                        for b in range(B))
            assert math.isclose(float(total), H * sum(seen), rel_tol=1e-3)


# ---------------------------------------------------------------------------
# what only the device can see
# ---------------------------------------------------------------------------
def device_status():
    return gqa.gqa_check_device_status(torch.cuda.current_stream())


BAD_LISTS = [
    ("negative past", dict(seqlens={1: -3}), gqa.GQA_ERR_INVALID_ARGUMENT),
    ("past beyond the bound", dict(seqlens={1: 220}), gqa.GQA_ERR_INVALID_ARGUMENT),
    ("past beyond the pages", dict(seqlens={1: 5000}), gqa.GQA_ERR_KV_OVERFLOW),
    ("huge past", dict(seqlens={1: 2**31 - 1}), gqa.GQA_ERR_KV_OVERFLOW),
]


@pytest.mark.parametrize("D,new", [(128, 1), (128, 40), (64, 3), (40, 2)])
@pytest.mark.parametrize("what,change,code", BAD_LISTS, ids=[x[0] for x in BAD_LISTS])
def test_a_bad_sequence_is_skipped(D, new, what, change, code):
    """It is reported, its rows stay as they are, the others are computed."""
    c = Case("bf16", H=8, Hkv=2, D=D, page=16, past=(60, 100, 31), new=(new, new, new), seed=3)
    c.table = torch.cat([c.table, torch.full((3, 8), -1, dtype=torch.int32)], 1)
    good = c.seqlens.clone()
    for b, v in change["seqlens"].items():
        c.seqlens[b] = v
    d = c.cuda()
    total = 200
    out, lse = run_attention(c, d, total=total)
    assert device_status() == code
    ro, rl, to, tl = ref_attention(c)
    rows = [r for b in (0, 2) for r in range(int(c.cu[b]), int(c.cu[b + 1]))]
    bad = list(range(int(c.cu[1]), int(c.cu[2])))
    assert_close(out[rows].view(len(rows), c.H, c.D), ro[rows], to[rows], what)
    assert (out[bad] == 7).all() and (lse[bad] == 7).all()
    assert device_status() == gqa.GQA_OK
    w0 = d["weights"].clone()
    gqa.paged_key_weights(d["query"], rl.nan_to_num(0.0).float().cuda(), d["k_pages"], d["weights"], d["table"],
                          d["cu"], d["seqlens"], new, total)
    assert device_status() == code
    mine = c.table[1, :7].long()
    assert same_bits(d["weights"][mine], w0[mine])
    k0 = d["k_pages"].clone()
    q = torch.full_like(d["query"], 7.0)
    gqa.paged_append(d["query"], d["key"], d["value"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["seqlens"],
                     total, query_out=q)
    assert device_status() == code
    assert (q[bad] == 7).all() and same_bits(d["k_pages"][mine], k0[mine])
    assert not same_bits(d["k_pages"][c.table[0, :4].long()], k0[c.table[0, :4].long()])
    # eviction looks at the cached tokens alone
    kept, left = gqa.paged_evict(d["k_pages"], d["v_pages"], d["weights"], d["table"], d["seqlens"], total, 20, 4)
    assert device_status() == code
    assert (kept[1] == -1).all() and left.tolist() == [20, change["seqlens"][1], 20]
    c.seqlens = good


@pytest.mark.parametrize("new", [1, 40])
def test_bad_row_lists(new):
    """cu_seqlens that run backwards, beyond the token arrays, or over the
    bound on new tokens."""
    base = Case("bf16", H=8, Hkv=2, D=128, page=16, past=(60, 100, 31), new=(new, new, new), seed=3)
    rows = base.query.shape[0]
    for cu in ([0, new, new - 1, 3 * new], [0, new, 2 * new, rows + 1], [-1, new, 2 * new, 3 * new],
               [0, new, 2 * new, -2**31], [0, -2**31, 2**31 - 1, 2**31 - 1]):
        d = base.cuda()
        d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out, lse = run_attention(base, d)
        assert device_status() == gqa.GQA_ERR_INVALID_ARGUMENT
        gqa.paged_key_weights(d["query"], lse, d["k_pages"], d["weights"], d["table"], d["cu"], d["seqlens"], new,
                              base.total)
        assert device_status() == gqa.GQA_ERR_INVALID_ARGUMENT
        gqa.paged_append(d["query"], d["key"], d["value"], d["k_pages"], d["v_pages"], d["table"], d["cu"],
                         d["seqlens"], base.total)
        assert device_status() == gqa.GQA_ERR_INVALID_ARGUMENT
    out, lse = run_attention(base, max_new=new, total=base.total)
    assert device_status() == gqa.GQA_OK


@pytest.mark.parametrize("D,new", [(128, 1), (128, 40), (64, 3), (40, 2)])
@pytest.mark.parametrize("entry", [-1, 2**31 - 1, -2**31, "num_pages"])
def test_bad_pages(D, new, entry):
    """A needed block-table entry outside the pool: reported, nothing read or
    written through it, the other sequences computed."""
    c = Case("fp16", H=8, Hkv=2, D=D, page=16, past=(60, 100, 31), new=(new, new, new), seed=3)
    ro, rl, to, tl = ref_attention(c)
    c.table[1, 3] = c.num_pages if entry == "num_pages" else entry
    c.table[1, 100 // 16] = c.table[1, 3]
    d = c.cuda()
    out, lse = run_attention(c, d)
    assert device_status() == gqa.GQA_ERR_INVALID_ARGUMENT
    rows = [r for b in (0, 2) for r in range(int(c.cu[b]), int(c.cu[b + 1]))]
    assert_close(out[rows].view(len(rows), c.H, c.D), ro[rows], to[rows], "others")
    gqa.paged_key_weights(d["query"], rl.nan_to_num(0.0).float().cuda(), d["k_pages"], d["weights"], d["table"],
                          d["cu"], d["seqlens"], new, c.total)
    assert device_status() == gqa.GQA_ERR_INVALID_ARGUMENT
    gqa.paged_append(d["query"], d["key"], d["value"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["seqlens"],
                     c.total)
    assert device_status() == gqa.GQA_ERR_INVALID_ARGUMENT
    gqa.paged_evict(d["k_pages"], d["v_pages"], d["weights"], d["table"], d["seqlens"], c.total, 50, 10)
    assert device_status() == gqa.GQA_ERR_INVALID_ARGUMENT


def test_bad_positions_and_destinations():
    c = Case("bf16", H=4, Hkv=2, D=64, page=16, past=(30, 5), new=(2, 2), seed=5, fill_new=False)
    cos, sin = caches(40, 64, "bf16")
    pos = torch.tensor([0, 40, -1, 39, 0, 0, 0], dtype=torch.int32)
    d = c.cuda()
    q = torch.full_like(d["query"], 7.0)
    gqa.paged_append(d["query"], d["key"], d["value"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["seqlens"],
                     c.total, cos_cache=cos.cuda(), sin_cache=sin.cuda(), positions=pos.cuda(), query_out=q)
    assert device_status() == gqa.GQA_ERR_INVALID_ARGUMENT
    assert (q[1] == 7).all() and (q[2] == 7).all() and not (q[0] == 7).all() and not (q[3] == 7).all()
    assert torch.isnan(d["k_pages"][int(c.table[0, 1]), :, 31 % 16].float()).all()
    # the kept tokens do not fit the destination's pages
    dst = c.free[:2].view(2, 1).cuda()
    kept, left = gqa.paged_evict(d["k_pages"], d["v_pages"], d["weights"], d["table"], d["seqlens"], c.total, 20, 4,
                                 dst_block_table=dst)
    assert device_status() == gqa.GQA_ERR_KV_OVERFLOW
    assert (kept[0] == -1).all() and left.tolist() == [30, 5] and kept[1, 0, :5].tolist() == [0, 1, 2, 3, 4]


# ---------------------------------------------------------------------------
# streams, graphs, workspaces
# ---------------------------------------------------------------------------
def step_case(new, seed, dtype="bf16"):
    return Case(dtype, H=8, Hkv=2, D=128, page=16, past=(300, 0, 1900), new=(new, new, 1), seed=seed)


@pytest.mark.parametrize("new", [1, 60])
def test_capture_and_replay_with_other_lengths(new):
    """A whole step captured once, replayed with other lists, lengths and rows;
    another graph and eager calls with the same Workspace in between."""
    ws = gqa.Workspace()
    cases = [step_case(new, 1), step_case(new, 2)]
    cases[1].past = [17, 600, 255]
    cases[1] = Case("bf16", H=8, Hkv=2, D=128, page=16, past=(17, 600, 255), new=(1, new, new), seed=2)
    rows = max(c.query.shape[0] for c in cases)
    pages = max(c.num_pages for c in cases)
    cols = max(c.table.shape[1] for c in cases)

    def padded(c):
        d = c.cuda()
        pad = lambda x, n: torch.cat([x, torch.zeros((n - x.shape[0],) + x.shape[1:], dtype=x.dtype, device="cuda")])  # noqa: E731
        for n in ("query", "key", "value"):
            d[n] = pad(d[n], rows)
        for n in ("k_pages", "v_pages", "weights"):
            d[n] = pad(d[n], pages)
        t = torch.full((c.B, cols), -1, dtype=torch.int32, device="cuda")
        t[:, :c.table.shape[1]] = d["table"]
        d["table"] = t
        return d

    def buffers():
        d = padded(cases[0])
        d["q"], d["out"] = torch.empty_like(d["query"]), torch.empty_like(d["query"])
        d["lse"] = torch.empty(rows, 8, device="cuda")
        d["w"] = torch.zeros_like(d["weights"])
        return d

    def step(d):
        lists = (d["table"], d["cu"], d["seqlens"])
        gqa.paged_append(d["query"], d["key"], d["value"], d["k_pages"], d["v_pages"], *lists, 1930, query_out=d["q"])
        gqa.paged_attention(d["q"], d["k_pages"], d["v_pages"], *lists, new, 1930, output=d["out"], lse=d["lse"],
                            workspace=ws)
        gqa.paged_key_weights(d["q"], d["lse"], d["k_pages"], d["w"], *lists, new, 1930, weights_in=d["weights"],
                              workspace=ws)

    graphs = []
    for _ in range(2):
        d = buffers()
        step(d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(d)
        graphs.append((g, d))

    def check(d, c):
        ok()
        n = c.tokens
        kp, vp = d["k_pages"].cpu()[:c.num_pages], d["v_pages"].cpu()[:c.num_pages]
        ro, rl, to, tl = ref_attention(c, kp, vp)
        assert same_bits(d["q"][:n], c.query[:n])
        assert_close(d["out"][:n].view(n, c.H, c.D), ro[:n], to[:n], "output")
        assert_close(d["lse"][:n], rl[:n], tl[:n], "lse")
        rw, tw, written = ref_weights(c, d["lse"].cpu()[:c.query.shape[0]], k_pages=kp)
        assert_close(d["w"].cpu()[:c.num_pages][written], rw[written], tw[written], "weights")

    for c in (cases[1], cases[0], cases[1]):
        for g, d in graphs:
            for n, x in padded(c).items():
                d[n].copy_(x)
            g.replay()
            check(d, c)
        eager = buffers()
        for n, x in padded(c).items():
            eager[n].copy_(x)
        step(eager)
        check(eager, c)
    # two graphs at once, on streams of their own: their scratch is not shared
    for n, x in padded(cases[0]).items():
        graphs[0][1][n].copy_(x)
    for n, x in padded(cases[1]).items():
        graphs[1][1][n].copy_(x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    check(graphs[0][1], cases[0])
    check(graphs[1][1], cases[1])


@pytest.mark.parametrize("new", [1, 60])
def test_two_streams_with_one_workspace(new):
    ws = gqa.Workspace()
    cases = [step_case(new, 1), step_case(new, 2, "fp16")]
    ds = [c.cuda() for c in cases]
    outs = [torch.empty_like(d["query"]) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for c, d, o, s in zip(cases, ds, outs, streams):
            gqa.paged_attention(d["query"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["seqlens"], new, c.total,
                                output=o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    ok()
    for c, o in zip(cases, outs):
        ro, _, to, _ = ref_attention(c)
        assert_close(o[:c.tokens].view(c.tokens, c.H, c.D), ro[:c.tokens], to[:c.tokens], "output")


def test_outputs_made_on_the_calls_stream():
    """stream= another than the current one, outputs and scratch left to the
    call."""
    c = step_case(60, 1)
    d = c.cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = gqa.paged_attention(d["query"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["seqlens"], 60, c.total,
                              stream=s)
    kept, left = gqa.paged_evict(d["k_pages"], d["v_pages"], d["weights"], d["table"], d["seqlens"], c.total, 100, 9,
                                 stream=s)
    s.synchronize()
    ok()
    ro, _, to, _ = ref_attention(c)
    assert_close(out[:c.tokens].view(c.tokens, c.H, c.D), ro[:c.tokens], to[:c.tokens], "output")
    assert left.tolist() == [100, 0, 100]


def test_refusals_name_the_tensor():
    c = step_case(1, 1)
    d = c.cuda()
    a = dict(query=d["query"], k_pages=d["k_pages"], v_pages=d["v_pages"], block_table=d["table"], cu_seqlens=d["cu"],
             seqlens_k=d["seqlens"], max_new_tokens=1, total_sequence_length=c.total)
    for name, bad in [("v_pages", d["v_pages"][:-1]), ("query", d["query"].float()), ("block_table", d["table"].long()),
                      ("cu_seqlens", d["cu"][:-1]), ("seqlens_k", d["seqlens"].cpu()),
                      ("query", d["query"].t().contiguous().t()), ("output", d["query"][:-1]),
                      ("lse", torch.empty(3, 3, device="cuda"))]:
        with pytest.raises(ValueError, match=name):
            gqa.paged_attention(**{**a, name: bad})
    with pytest.raises(gqa.GqaError) as e:
        gqa.paged_attention(**{**a, "total_sequence_length": 10**6})
    assert e.value.status == gqa.GQA_ERR_KV_OVERFLOW
    with pytest.raises(gqa.GqaError) as e:
        gqa.paged_attention(**{**a, "output": d["query"]})
    assert e.value.status == gqa.GQA_ERR_INVALID_ARGUMENT
    with pytest.raises(ValueError, match="weights"):
        gqa.paged_evict(d["k_pages"], d["v_pages"], d["weights"][..., :-1], d["table"], d["seqlens"], c.total, 10, 0)
    with pytest.raises(gqa.GqaError):
        gqa.paged_evict(d["k_pages"], d["v_pages"], d["weights"], d["table"], d["seqlens"], c.total, 10, 11)
    ok()


def test_scratch_of_a_captured_stream_that_is_not_current():
    """A call on a captured stream keeps scratch of its own, whatever the
    current stream."""
    c = Case("fp16", H=8, Hkv=1, D=64, page=16, past=(700, 90), new=(1, 1), seed=21)
    d = c.cuda()
    args = [d[x] for x in ("query", "k_pages", "v_pages", "table", "cu", "seqlens")]
    ws = gqa.Workspace()
    want = gqa.paged_attention(*args, c.max_new, c.total, workspace=ws)[:c.tokens]
    buffers = len(ws.paged)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = gqa.paged_attention(*args, c.max_new, c.total, workspace=ws, stream=side)[:c.tokens]
    assert len(ws.paged) == buffers
    graph.replay()
    ok()
    assert same_bits(got, want)


@pytest.mark.parametrize("new", [5, 6, 8])  # 20, 24 and 32 rows a KV head
@pytest.mark.parametrize("total", [1000, 1536, 5120])
def test_attention_of_few_rows_over_much_work(new, total):
    """Lengths on both sides of where few rows of head size 128 go to the chunk
    kernel (64 KV heads in the batch)."""
    g = torch.Generator().manual_seed(total + new)
    past = [int(torch.randint(0, 700, (1,), generator=g)) for _ in range(8)]
    past[0] = 900
    c = Case("bf16", H=32, Hkv=8, D=128, page=32, past=past, new=(new, 1, new, 0, 2, new, new, 3), seed=total)
    pad = -(-total // 32) - c.table.shape[1]
    c.table = torch.cat([c.table, torch.full((8, max(pad, 0)), -1, dtype=torch.int32)], 1)
    check_attention(c, total=total)


@pytest.mark.parametrize("D,dtype", [(8, "fp16"), (72, "bf16"), (136, "fp16"), (256, "bf16")])
@pytest.mark.parametrize("window", [0, 600])
def test_attention_of_other_head_sizes_over_long_pasts(D, dtype, window):
    """Few rows over many slots, where several CTAs share a row."""
    check_attention(Case(dtype, H=6, Hkv=2, D=D, page=16, past=(3000, 0, 31, 1023), new=(1, 2, 0, 3), window=window,
                         seed=D))
