"""GPU tests of the attention operators at values and masks where one key, row or element must not reach another:
zero and tiny scores, cache contents that no row sees, extreme windows and queries, copied elements."""
import math

import numpy as np
import pytest
import torch

from test_gpu_attention import DT, STEP, build_cache, check, gen, reference, w4  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def packed(bits):
    """Truth values [T, 32 * words] as a draft mask's words."""
    return torch.from_numpy(np.packbits(bits.cpu().numpy(), axis=1, bitorder="little").view(np.int32).copy()).cuda()


def tree_bits(T, words, seed):
    return torch.rand(T, 32 * words, generator=gen(seed), device="cuda") < 0.4


# ---- scores whose factor leaves float32's range (zero queries, zero or tiny keys)

@pytest.mark.parametrize("kind", ["zero keys", "tiny keys", "all zero", "some zero queries"])
@pytest.mark.parametrize("form", ["causal", "window", "tree"])
@pytest.mark.parametrize("n,G,D,kv", [(40, 8, 128, 300), (70, 1, 64, 77), (33, 4, 128, 33), (300, 2, 64, 401)])
def test_many_rows_of_zero_scores(w4, n, G, D, kv, form, kind):
    """Zero queries and zero or tiny keys: every visible key weighs the same, hidden ones nothing."""
    Hkv, page = 2, 16
    g = gen(n + kv)
    k, v = torch.randn(2, kv, Hkv, D, generator=g, device="cuda")
    if kind != "some zero queries":
        k *= 2.0 ** -40 if kind == "tiny keys" else 0.0
    if kind == "all zero":
        v *= 0
    q = torch.randn(n, Hkv * G, D, generator=g, device="cuda").to(torch.bfloat16)
    if kind == "some zero queries":
        q[::3] = 0
        k[: kv // 2] = 0                     # whole tiles of zero keys beside others
    else:
        q *= 0
    pages = -(-kv // page)
    cache = torch.full((pages, Hkv, page * (D + D // 8)), 255, dtype=torch.uint8, device="cuda")
    slots = torch.arange(kv, device="cuda")
    w4.w4a16_kv_append(cache, k, v, slots)
    gk, gv = (x.double() for x in w4.w4a16_kv_read(cache, slots, D))
    bits = tree_bits(n, -(-n // 32), 3) if form == "tree" else None
    window = 29 if form == "window" else 0
    lse = torch.full((n, Hkv * G), 3.0, device="cuda")
    got = w4.w4a16_attention(q, cache, torch.arange(pages, dtype=torch.int32, device="cuda")[None], i32(kv), i32(0, n),
                             max_q=n, scale=0.088, window=window, tree_mask=None if bits is None else packed(bits), lse=lse)
    assert w4.w4a16_device_error() == 0
    check(q, got, lse, reference(q, [gk], [gv], [n], [kv], float(np.float32(0.088)), True, window, bits), "bf16")


# ---- memory taken by a call on another stream

@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("n", [1, 40])
def test_side_stream_has_memory_of_its_own(w4, n, raw):
    """On a stream that is still busy, without workspace and out: what the current stream allocates and writes in the
    meantime is other memory, and the call's results stay after it."""
    cache, bt, _, _ = build_cache([3000, 700], 2, 128, 64, 4)
    q = torch.randn(2 * n, 16, 128, generator=gen(3), device="cuda").to(torch.bfloat16)
    args = (cache, bt, i32(3000, 700), i32(0, n, 2 * n))
    pos, tab = torch.arange(2 * n, dtype=torch.int32, device="cuda"), w4.w4a16_rope_table(2 * n, 128)
    slots = bt[0, :5].long() * 64
    want = w4.w4a16_attention(q, *args, max_q=n, scale=0.1), w4.w4a16_rope(q, pos, tab), *w4.w4a16_kv_read(cache, slots, 128)
    need = w4.w4a16_attention_workspace_size(2 * n, 2, 2, 8, 128, n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    on = s.cuda_stream if raw else s
    got = (w4.w4a16_attention(q, *args, max_q=n, scale=0.1, stream=on), w4.w4a16_rope(q, pos, tab, stream=on),
           *w4.w4a16_kv_read(cache, slots, 128, stream=on))
    other = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all((o == 255).all() for o in other) and w4.w4a16_device_error() == 0


# ---- what the cache and the block table hold at keys that no row sees

def poison(cache, bt, page, D, b, keys, scale_bits):
    """Codes of all ones and the given bf16 scale bits at the places of a sequence's keys."""
    blocks = cache.view(cache.shape[0], cache.shape[1], page // 16, -1)
    at = (bt[b].long()[keys // page][:, None], torch.arange(cache.shape[1], device="cuda")[None],
          (keys % page // 16)[:, None], (keys % 16)[:, None])
    for part in (0, 1):
        blocks[..., part * 8 * D:(part + 1) * 8 * D].unflatten(-1, (16, D // 2))[at] = 255
        scales = blocks[..., 16 * D + part * D:16 * D + (part + 1) * D].unflatten(-1, (16, D // 16))
        scales[at] = torch.tensor([scale_bits & 255, scale_bits >> 8] * (D // 32), dtype=torch.uint8, device="cuda")


JUNK = [0xFFFF, 0x7F80, 0x7F00, 0x5F00]   # NaN, infinity, 2^127, 2^63


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs,Hkv,G,D,page,window", [
    ([(1, 2000), (1, 40)], 2, 8, 128, 16, 50), ([(1, 333)], 1, 4, 64, 64, 1), ([(1, 700)], 1, 5, 256, 32, 33),
    ([(40, 1500), (3, 200)], 2, 8, 128, 16, 100), ([(70, 900)], 1, 2, 64, 16, 7), ([(300, 1111)], 1, 4, 128, 32, 130),
    ([(9, 129), (33, 257)], 2, 16, 64, 16, 1),
])
def test_nothing_behind_the_window_is_looked_at(w4, seqs, Hkv, G, D, page, window, dtype):
    """Pages wholly behind every row's window may be gone from the block table, and hidden tokens of the page at
    the border may be anything."""
    ns, kvs = [s[0] for s in seqs], [s[1] for s in seqs]
    cache, bt, keys, values = build_cache(kvs, Hkv, D, page, 5)
    q = torch.randn(sum(ns), Hkv * G, D, generator=gen(8), device="cuda").to(DT[dtype])
    starts = i32(0, *np.cumsum(ns).tolist())
    kw = dict(max_q=max(ns), scale=0.1, window=window)
    lse = torch.empty(sum(ns), Hkv * G, device="cuda")
    want = w4.w4a16_attention(q, cache, bt, i32(*kvs), starts, lse=lse, **kw)
    check(q, want, lse, reference(q, keys, values, ns, kvs, float(np.float32(0.1)), True, window, None), dtype)
    for junk in JUNK:
        bad, table = cache.clone(), bt.clone()
        for b, (n, kv) in enumerate(seqs):
            lo = max(0, kv - n + 1 - window)
            poison(bad, bt, page, D, b, torch.arange(lo, device="cuda"), junk)
            # gone, or (every other page) an entry that was never written
            table[b, :lo // page] = -1
            table[b, 1:lo // page:2] = bt[b, 1:lo // page:2]
        got = w4.w4a16_attention(q, bad, table, i32(*kvs), starts, **kw)
        assert w4.w4a16_device_error() == 0
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs,Hkv,G,D,page,real", [
    ([(16, 900), (16, 16), (16, 333)], 2, 8, 128, 32, 7), ([(2, 40)], 1, 4, 64, 16, 1), ([(64, 500)], 1, 8, 128, 64, 33),
    ([(100, 130)], 1, 1, 64, 16, 40), ([(40, 300), (5, 90)], 1, 2, 256, 32, 3), ([(150, 700)], 2, 4, 128, 16, 100),
    ([(40, 30)], 1, 8, 128, 16, 20),
])
def test_drafts_that_no_row_sees(w4, seqs, Hkv, G, D, page, real, dtype):
    """A tree padded to a fixed size: the places of drafts that no row's mask shows may be anything."""
    ns, kvs = [s[0] for s in seqs], [s[1] for s in seqs]
    T, words = sum(ns), -(-max(ns) // 32)
    cache, bt, keys, values = build_cache(kvs, Hkv, D, page, 5)
    q = torch.randn(T, Hkv * G, D, generator=gen(8), device="cuda").to(DT[dtype])
    starts = i32(0, *np.cumsum(ns).tolist())
    bits = tree_bits(T, words, 4)
    bits[:, real:] = False                  # drafts from `real` on are padding,
    bits[:, real // 2] = False              # and one in the middle is seen by nobody
    kw = dict(max_q=max(ns), scale=0.1, tree_mask=packed(bits))
    lse = torch.empty(T, Hkv * G, device="cuda")
    want = w4.w4a16_attention(q, cache, bt, i32(*kvs), starts, lse=lse, **kw)
    check(q, want, lse, reference(q, keys, values, ns, kvs, float(np.float32(0.1)), True, 0, bits), dtype)
    for junk in JUNK:
        bad = cache.clone()
        for b, (n, kv) in enumerate(seqs):
            d = torch.arange(n, device="cuda")
            d = d[((d >= real) | (d == real // 2)) & (kv - n + d >= 0)]
            poison(bad, bt, page, D, b, kv - n + d, junk)
        got = w4.w4a16_attention(q, bad, bt, i32(*kvs), starts, **kw)
        assert w4.w4a16_device_error() == 0
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,kv", [(40, 3), (300, 120), (5, 2), (1, 50)])
def test_largest_window_is_no_window(w4, n, kv, dtype):
    """The largest window an int holds, also where query tokens stand before the first key."""
    cache, bt, keys, values = build_cache([kv], 1, 128, 16, 5)
    q = torch.randn(n, 8, 128, generator=gen(8), device="cuda").to(DT[dtype])
    args = (q, cache, bt, i32(kv), i32(0, n))
    lse, lse2 = torch.empty(2, n, 8, device="cuda")
    want = w4.w4a16_attention(*args, max_q=n, scale=0.1, lse=lse)
    check(q, want, lse, reference(q, keys, values, [n], [kv], float(np.float32(0.1)), True, 0, None), dtype)
    for window in (2 ** 31 - 1, 2 ** 31 - n, 2 ** 30):
        got = w4.w4a16_attention(*args, max_q=n, scale=0.1, window=window, lse=lse2)
        assert torch.equal(got, want) and torch.equal(lse, lse2)
    assert w4.w4a16_device_error() == 0


# ---- rotation: elements that are copied

def bits_of(x):
    return x.contiguous().view(torch.int32 if x.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 64), (128, 20), (64, 18), (72, 40), (64, 64), (128, 2)])
def test_rope_copies_are_copies(w4, D, rot, interleaved, dtype):
    """Dims from rot on, and whole tokens whose position is outside the table, come through bit for bit: infinities
    and signed zeros beside other values too."""
    T, H, P = 9, 5, 50
    x = torch.randn(T, H, D, generator=gen(D + rot), device="cuda").to(DT[dtype])
    odd = torch.tensor([math.inf, 1.0, -math.inf, 0.0, -0.0, -2.0, 3.0, -0.0], device="cuda").to(DT[dtype])
    x[..., rot:] = odd.repeat(D // 8 + 1)[:D - rot]
    pos = torch.randint(0, P, (T,), generator=gen(2), device="cuda", dtype=torch.int32)
    bad = torch.tensor([2, 5], device="cuda")
    pos[2], pos[5] = -1, P
    x[bad] = odd.repeat(D // 8)
    tab = w4.w4a16_rope_table(P, rot)
    for inverse in (False, True):
        y = w4.w4a16_rope(x, pos, tab, interleaved=interleaved, inverse=inverse)
        assert w4.w4a16_device_error() == 1
        assert torch.equal(bits_of(y[bad]), bits_of(x[bad]))
        assert torch.equal(bits_of(y[..., rot:]), bits_of(x[..., rot:]))
        assert torch.isfinite(y[0, :, :rot]).all()


# ---- queries near the largest number

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("e", [100, 119, 122, 124, 126])
def test_huge_queries(w4, n, e, dtype):
    """Queries of 2^e with scores inside float32's range: one key takes all the weight; over zero keys all weigh the
    same."""
    G, D, page, kv = 8, 128, 16, 20 + n
    cache, bt, keys, values = build_cache([kv], 1, D, page, 6)
    q = torch.zeros(n, G, D, device="cuda")
    q[..., 5] = 2.0 ** e
    q = q.to(DT[dtype])
    lse = torch.empty(n, G, device="cuda")
    args = (i32(kv), i32(0, n))
    got = w4.w4a16_attention(q, cache, bt, *args, max_q=n, scale=0.01, lse=lse, causal=False)
    top = keys[0][:, 0, 5].topk(2).values
    assert (top[0] - top[1]) * 0.01 * 2.0 ** e > 2.0 ** 20           # (the others weigh nothing)
    best = keys[0][:, 0, 5].argmax()
    # weights are exact (one key), the output is rounded to the type; exp2, sums and the quotient: a few 2^-23
    want = values[0][best, 0].expand(n, G, D)
    assert ((got.double() - want).abs() <= want.abs() * (STEP[dtype] * (1 + 2.0 ** -6) + 2.0 ** -20)).all()
    score = top[0] * float(np.float32(0.01)) * 2.0 ** e
    assert ((lse.double() - score).abs() <= score * 2.0 ** -20).all()
    k = torch.zeros(kv, 1, D, device="cuda")
    zero = torch.full_like(cache, 255)
    slots = bt[0].long()[torch.arange(kv, device="cuda") // page] * page + torch.arange(kv, device="cuda") % page
    w4.w4a16_kv_append(zero, k, torch.randn(kv, 1, D, generator=gen(3), device="cuda"), slots)
    got = w4.w4a16_attention(q, zero, bt, *args, max_q=n, scale=0.01, lse=lse, causal=False)
    v = w4.w4a16_kv_read(zero, slots, D)[1].double()
    check(q, got, lse, reference(q, [k.double()], [v], [n], [kv], 0.01, False, 0, None), dtype)
    assert w4.w4a16_device_error() == 0
