"""lora_prompt_attention and lora_prefix_attention against a 64-bit reference."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L
from attn_util import Batch

pytestmark = pytest.mark.gpu


def go(*a, **kw):
    b = Batch(*a, **kw).upload()
    b.run()
    b.check()
    return b


@pytest.mark.parametrize("heads", [(1, 1, 128), (2, 2, 64), (4, 1, 128), (6, 2, 64), (7, 1, 128), (10, 2, 96),
                                   (16, 2, 40), (3, 1, 8), (64, 1, 64), (128, 1, 16)])
@pytest.mark.parametrize("page", [0, 16])
def test_heads_and_sizes(heads, page):
    # whole prompts of lengths around one token, a block of keys and a tile of queries, one behind cached keys
    go([1, 5, 127, 130, 33], [1, 5, 127, 130, 90], heads=heads, page=page, seed=1)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384, 511, 700])
def test_one_prompt_of_every_kind_of_length(n):
    go([n], [n], heads=(4, 1, 64), seed=n)


@pytest.mark.parametrize("n", [1, 7, 8, 127, 128, 129, 256, 511, 512, 513, 1000, 3000])
@pytest.mark.parametrize("page", [0, 32])
def test_single_tokens(n, page):
    go([1, 1, 1], [n, 1, max(1, n // 2)], heads=(8, 2, 128), page=page, seed=n)


@pytest.mark.parametrize("page", [8, 16, 24, 48, 64, 128, 192, 256])
def test_pages(page):
    go([1, 40, 200], [page + 1, 300, 2 * page + 200], heads=(4, 2, 128), page=page, seed=page)


def test_rows_that_see_no_key():
    # more queries than keys (the first rows see none), no keys at all, and no queries
    b = go([5, 3, 0, 200, 1], [2, 0, 40, 130, 0], heads=(4, 2, 64), seed=3)
    out = b.out.float().cpu()
    assert torch.all(out[0:3] == 0) and torch.all(out[5:8] == 0) and torch.all(out[8:8 + 70] == 0)
    assert torch.all(out[208] == 0)


def test_not_causal():
    go([3, 150, 1, 9], [200, 150, 77, 0], heads=(6, 3, 64), causal=0, seed=4)


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf"), -3.3895e38])
@pytest.mark.parametrize("page", [0, 16])
def test_rows_of_nobody_do_not_matter(poison, page):
    go([1, 70, 3], [130, 200, 129], heads=(4, 2, 128), page=page, poison=poison, seed=5)


def test_strides():
    go([17, 140], [60, 140], heads=(4, 2, 64), q_pad=72, kv_pad=24, out_pad=40, seed=6)


def test_packed_qkv_rows():
    """Queries, keys and values as columns of one tensor, the output of a QKV layer."""
    hq, hkv, d = 4, 2, 64
    b = Batch([50, 1, 170], [50, 1, 170], heads=(hq, hkv, d), seed=7).upload()
    qkv = torch.full((b.T, (hq + 2 * hkv) * d), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], 1)
    q.copy_(b.dq)
    rows = torch.cat(b.place).cuda()
    k.copy_(b.dk[rows])
    v.copy_(b.dv[rows])
    b.dq, b.dk, b.dv = q, k, v
    b.dtable = b.dcu[:-1].reshape(-1, 1)
    b.run()
    b.check()


def test_large_scores():
    # one key takes nearly all the weight, and the running maximum moves by more than any fixed allowance
    b = Batch([300], [300], heads=(2, 1, 128), spread=4.0, seed=8)
    b.k[b.place[0], :] *= torch.linspace(0.1, 3.0, 300)[:, None].to(torch.bfloat16)
    b.upload().run()
    b.check()


def test_a_score_far_below_the_rest_does_not_vanish_into_nan():
    b = Batch([40], [40], heads=(2, 1, 64), seed=9)
    b.k[b.place[0][:7], :] = -1e30
    b.q[:, :] = b.q.abs()
    b.upload().run()
    b.check()


@pytest.mark.parametrize("heads", [(4, 1, 128), (6, 2, 64), (8, 8, 64), (28, 4, 128)])
@pytest.mark.parametrize("page", [0, 16])
def test_prefixes(heads, page):
    go([1, 1, 3, 1, 1, 40, 1], [1, 30, 3, 129, 0, 90, 7], heads=heads, page=page, groups=[0, 3, 3, 4, 7],
       prefix_lens=[130, 500, 0, 1], seed=10)


@pytest.mark.parametrize("plen", [1, 127, 128, 129, 513, 2000])
def test_one_prefix_for_all(plen):
    go([1] * 70, list(range(70)), heads=(8, 2, 64), page=32, groups=[0, 70], prefix_lens=[plen], seed=plen)


def test_prefix_of_no_keys_and_own_keys_none():
    b = go([2, 1, 1], [0, 0, 5], heads=(4, 2, 64), page=16, groups=[0, 1, 2, 3], prefix_lens=[0, 20, 0], seed=11)
    assert torch.all(b.out[:2] == 0)


def test_split_over_keys_and_repeatable():
    """Few rows and many keys: ranges of keys are joined, the same way every time."""
    b = Batch([1, 2], [20000, 9000], heads=(4, 2, 128), page=64, seed=12).upload()
    b.run()
    first = b.out.clone()
    for _ in range(3):
        b.out.fill_(7.0)
        b.run()
        assert torch.equal(b.out.view(torch.int16), first.view(torch.int16))
    b.check()


@pytest.mark.parametrize("heads", [(7, 1, 128), (14, 2, 72), (3, 3, 24), (12, 2, 64), (8, 8, 64)])
@pytest.mark.parametrize("tokens", [3, 100, 300])
def test_joins_of_few_and_many_tokens(heads, tokens):
    """Partial results of every batch size, in a workspace that begins on 16 bytes and ends where it says."""
    b = Batch([1] * (tokens - 2) + [2], [i % 50 for i in range(tokens - 1)], heads=heads, page=16,
              groups=[0, tokens - 1], prefix_lens=[4500 if tokens == 3 else 900], seed=tokens).upload()
    whole = torch.full((b.ws_bytes + 16 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    whole[16:16 + b.ws_bytes] = 0
    b.ws = whole[16:16 + b.ws_bytes]
    assert b.ws.data_ptr() % 32 == 16
    b.run()
    b.check()
    assert torch.all(whole[:16] == 0xA5) and torch.all(whole[16 + b.ws_bytes:] == 0xA5)


def test_long_prompt():
    b = Batch([1500], [1500], heads=(4, 1, 128), seed=13).upload()
    b.run()
    b.check()


def test_one_plan_for_batches_of_different_sizes():
    big = Batch([30, 200, 1], [30, 260, 900], heads=(4, 2, 64), page=16, seed=14).upload()
    big.run()
    big.check()
    small = Batch([2, 1], [17, 4], heads=(4, 2, 64), page=16, seed=15).upload()
    small.plan, small.ws, small.ws_bytes = big.plan, big.ws, big.ws_bytes
    small.build()
    small.run()
    small.check()
    big.build()
    big.run()
    big.check()


def test_another_stream_and_a_graph():
    b = Batch([1, 1, 30], [600, 40, 700], heads=(4, 2, 128), page=16, seed=16).upload()
    ref = b.reference()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b.build()
        b.run()
    s.synchronize()
    b.check(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.build()
        b.run()
    b.out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    b.check(ref)


def test_cache_past_32_bit_offsets():
    """Rows whose element offset is past 2^31 (and byte offset past 2^32)."""
    d, hkv, first = 128, 8, (1 << 21) + 1024
    b = Batch([1, 20], [300, 90], heads=(16, hkv, d), page=16, seed=17, first_row=first)
    k, v = b.k, b.v
    b.upload()
    b.dk = torch.empty((b.rows, hkv * d), dtype=torch.bfloat16, device="cuda")
    b.dv = torch.empty_like(b.dk)
    b.dk[first:], b.dv[first:] = k.cuda(), v.cuda()
    b.run()
    b.check()


def test_bad_lengths_leave_the_output_alone():
    for spoil in ("cu_down", "cu_end", "cu_start", "kv_negative", "kv_too_long"):
        b = Batch([4, 3], [10, 9], heads=(4, 2, 64), seed=18).upload()
        if spoil == "cu_down":
            b.dcu[1] = 9
        elif spoil == "cu_end":
            b.dcu[2] = 6
        elif spoil == "cu_start":
            b.dcu[0] = 1
        elif spoil == "kv_negative":
            b.dkv[1] = -1
        else:
            b.dkv[0] = 11
        b.out.fill_(7.0)
        b.build()
        b.run()
        assert L.lora_attn_get_status(b.plan) == L.CODE["LORA_ERR_DEVICE_INDEX"], spoil
        assert L.lora_attn_get_status(b.plan) == 0
        assert torch.all(b.out == 7.0), spoil
    for spoil in ("down", "end", "long"):
        b = Batch([1, 1], [3, 3], heads=(4, 2, 64), seed=18, groups=[0, 1, 2], prefix_lens=[5, 6]).upload()
        if spoil == "down":
            b.dgs[1] = 3
        elif spoil == "end":
            b.dgs[2] = 1
        else:
            b.dpl[0] = 7
        b.out.fill_(7.0)
        b.build()
        b.run()
        assert L.lora_attn_get_status(b.plan) == L.CODE["LORA_ERR_DEVICE_INDEX"], spoil
        assert torch.all(b.out == 7.0), spoil


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("wild", [-5, 1 << 30, 2147483647, -2147483648])
def test_table_entries_outside_the_cache(page, wild):
    """Such rows count as zero keys and values and the status says so; the other sequence is not touched."""
    b = Batch([1, 1], [40, 40], heads=(4, 2, 64), page=page, seed=19, poison=0.5).upload()
    ref = b.reference()
    b.dtable[0, 0] = wild
    b.run()
    assert L.lora_attn_get_status(b.plan) == L.CODE["LORA_ERR_DEVICE_INDEX"]
    got = b.out.float().cpu().double().view(2, 4, 64)
    # the rows that the spoilt line leads to; zeros in the place of those outside
    rows = b.place[0].clone()
    moved = 16 if page else 40
    rows[:moved] = wild * (page or 1) + torch.arange(moved)
    outside = (rows < 0) | (rows >= b.rows)
    assert outside.any()
    at = rows.clamp(0, b.rows - 1)
    k, v = b.k[at], b.v[at]
    k[outside], v[outside] = 0, 0
    z = Batch([1, 1], [40, 40], heads=(4, 2, 64), page=page, seed=19)
    z.k[z.place[0]], z.v[z.place[0]] = k, v
    ref0, mag0 = z.reference()
    assert torch.all((got[0] - ref0[0]).abs() <= 2.0 ** -7 * mag0[0] + 2.0 ** -8 * ref0[0].abs() + 1e-30)
    assert torch.all((got[1] - ref[0][1]).abs() <= 2.0 ** -7 * ref[1][1] + 2.0 ** -8 * ref[0][1].abs())


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("wild", [-5, 1 << 30, 2147483647, -2147483648])
def test_own_keys_outside_the_cache(page, wild):
    """The same for the few own keys of single tokens behind a prefix: the first sequence's all lie outside."""
    kw = dict(heads=(4, 2, 64), page=page, groups=[0, 2], prefix_lens=[30], seed=22, poison=0.5)
    b = Batch([1, 1], [9, 9], **kw).upload()
    ref = b.reference()
    b.dtable[0, 0] = wild if page or wild > 0 else -40
    b.run()
    assert L.lora_attn_get_status(b.plan) == L.CODE["LORA_ERR_DEVICE_INDEX"]
    got = b.out.float().cpu().double().view(2, 4, 64)
    z = Batch([1, 1], [9, 9], **kw)
    z.k[z.place[0]], z.v[z.place[0]] = 0, 0
    ref0, mag0 = z.reference()
    assert torch.all((got[0] - ref0[0]).abs() <= 2.0 ** -7 * mag0[0] + 2.0 ** -8 * ref0[0].abs() + 1e-30)
    assert torch.all((got[1] - ref[0][1]).abs() <= 2.0 ** -7 * ref[1][1] + 2.0 ** -8 * ref[0][1].abs())


@pytest.mark.parametrize("page", [0, 24, 64])
@pytest.mark.parametrize("heads", [(5, 1, 128), (8, 8, 64), (14, 2, 40), (2, 1, 8)])
@pytest.mark.parametrize("tokens", [5, 400])
def test_single_tokens_with_few_own_keys(tokens, heads, page):
    """Lengths around the number of own keys that need no item, with and without a prefix before them."""
    own = [(0, 1, 2, 7, 8, 15, 16, 17, 18, 31, 33)[i % 11] for i in range(tokens - 1)]
    b = go([1] * (tokens - 2) + [3, 1], own[:-1] + [3, 16], heads=heads, page=page,
           groups=[0, tokens // 2, tokens // 2, tokens], prefix_lens=[0, 5, 40], seed=tokens, q_pad=8, kv_pad=16, out_pad=8)
    assert torch.all(b.out[0, :heads[0] * heads[2]] == 0)  # no key at all


def refused(code, f):
    with pytest.raises(L.LoraError) as e:
        f()
    assert e.value.code == L.CODE[code], e.value


def test_refusals():
    b = Batch([4, 3], [10, 9], heads=(4, 2, 64), page=16, seed=20).upload()
    args = [b.plan, b.dq, b.dq.stride(0), b.dk, b.dk.stride(0), b.dv, b.dv.stride(0), b.dk.shape[0], b.dtable,
            b.dtable.stride(0), b.out, b.out.stride(0), b.ws, b.ws_bytes]

    def call(i, value):
        a = list(args)
        a[i] = value
        return lambda: L.lora_prompt_attention(*a)

    inv = "LORA_ERR_INVALID_ARG"
    for i in (1, 3, 5, 8, 10, 12):
        refused(inv, call(i, None))
    for i in (1, 3, 5, 10):
        refused(inv, call(i, args[i].data_ptr() + 2))
    refused(inv, call(8, args[8].data_ptr() + 2))
    for i, width in ((2, 256), (4, 128), (6, 128), (11, 256)):
        refused(inv, call(i, width - 8))
        refused(inv, call(i, width + 4))
    refused(inv, call(7, -1))
    refused(inv, call(9, 0))                       # a table too narrow for the longest sequence
    refused("LORA_ERR_CAPACITY", call(13, b.ws_bytes - 16))
    refused("LORA_ERR_UNSUPPORTED", lambda: L.lora_prefix_attention(*args[:10], b.dtable, 1, *args[10:]))
    g = Batch([1], [3], heads=(4, 2, 64), page=16, seed=20, groups=[0, 1], prefix_lens=[5]).upload()
    refused("LORA_ERR_UNSUPPORTED", lambda: L.lora_prompt_attention(g.plan, *args[1:]))
    refused(inv, lambda: L.lora_prefix_attention(g.plan, *args[1:10], None, 1, *args[10:12], g.ws, g.ws_bytes))
    fresh = L.AttnPlan()
    refused(inv, lambda: L.lora_prompt_attention(fresh, *args[1:]))
    size = L.lora_attn_plan_bytes(b.desc(), 8, 2, 0)
    buf = torch.empty(size, dtype=torch.uint8, device="cuda")
    L.lora_attn_plan_bind(fresh, b.desc(), buf, size, 8, 2, 0)
    refused(inv, lambda: L.lora_prompt_attention(fresh, *args[1:]))  # bound, nothing built
    refused("LORA_ERR_CAPACITY", lambda: L.lora_attn_plan_bind(fresh, b.desc(), buf, size - 1, 8, 2, 0))
    refused(inv, lambda: L.lora_attn_plan_bind(fresh, b.desc(), buf.data_ptr() + 4, size, 8, 2, 0))
    L.lora_attn_plan_bind(fresh, b.desc(), buf, size, 8, 2, 0)

    def build(n=2, t=7, cu=b.dcu, kv=b.dkv, g=0, gs=None, pl=None, mk=10, mp=0):
        return lambda: L.lora_attn_build_plan(fresh, n, t, cu, kv, g, gs, pl, mk, mp)

    refused("LORA_ERR_CAPACITY", build(n=3))
    refused("LORA_ERR_CAPACITY", build(t=9))
    refused("LORA_ERR_CAPACITY", build(g=1, gs=b.dcu, pl=b.dkv))
    refused(inv, build(cu=None))
    refused(inv, build(kv=None))
    refused(inv, build(n=-1))
    refused(inv, build(t=-1))
    refused(inv, build(mk=-1))
    refused(inv, build(mk=(1 << 30) + 1))
    refused(inv, build(mp=(1 << 30) + 1))
    for field, value in (("n_q_heads", 3), ("n_q_heads", 0), ("n_kv_heads", 0), ("head_dim", 12), ("head_dim", 136),
                         ("head_dim", 0), ("page_size", 12), ("page_size", -8), ("causal", 2), ("scale", 0.0),
                         ("scale", -1.0), ("scale", float("nan")), ("scale", float("inf"))):
        d = b.desc()
        setattr(d, field, value)
        assert L.lora_attn_plan_bytes(d, 8, 2, 0) == 0, field
        refused(inv, lambda: L.lora_attn_plan_bind(fresh, d, buf, size, 8, 2, 0))
    d = b.desc()
    d.n_q_heads, d.n_kv_heads = 129, 1
    assert L.lora_attn_plan_bytes(d, 8, 2, 0) == 0


def test_empty_batches():
    b = Batch([4], [10], heads=(4, 2, 64), seed=21).upload()
    b.T, b.n = 0, 0
    b.build()
    b.run()
    assert torch.all(b.out == 7.0)
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    L.lora_attn_build_plan(b.plan, 1, 0, z, z, 0, None, None, 0, 0)
    b.run()
    assert torch.all(b.out == 7.0)
    assert L.lora_attn_get_status(b.plan) == 0
