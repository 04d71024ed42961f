"""The 8-bit cache on the GPU, through the C ABI, against the float64 oracle: writing
(bit-exact), reading back (exact: the scales are powers of two), decode and chunked prefill.

Tolerances of decode and prefill are those of parity_util (1e-2 and one bf16 spacing on each
output, 1e-3 on the mean and on the LSE), against the oracle on the same codes. The kernel's
own roundings stay below them: q in 8-bit digits is off by at most 2^-22 of the row's largest
value, so a score of D = 128 products moves by at most 2^-22 * 128 * |q| |k| scale
< 2^-22 * 128 * 4 * 4 * 0.089 = 5e-5 in the worst case of equal signs and by 5e-7 for random ones;
P in two digits is off by at most 2^-9 of itself (E4M3) or 2^-16 (int8), which moves an output
of a weighted mean by at most 2^-9 of max|V - O| / 2 < 1e-2 for |V| < 5."""

import numpy as np
import pytest
import torch

import attention_online_softmax_fwd_b200 as ab
from attention_online_softmax_fwd_b200 import inputs as gen
from oracle import attn_oracle as orc
from parity_util import compare_output

pytestmark = pytest.mark.gpu

KINDS = ["e4m3", "int8"]


def to(dev, *ts):
    return [t.to(dev) for t in ts]


def quantized(cache, block, kind):
    kc, ks = gen.quantize_pool_q8(cache.k_pages, block, kind)
    vc, vs = gen.quantize_pool_q8(cache.v_pages, block, kind)
    return kc, vc, ks, vs


def empty_rows(o, lse, lens):
    for b, L in enumerate(lens):
        if L == 0:
            o[b], lse[b] = 0.0, -np.inf
    return o, lse


# ------------------------------------------------------------------ writing

def random_pool(g, P, page, block, Hkv, D, kind):
    if kind == "e4m3":
        codes = torch.randint(0, 256, (P, page, Hkv, D), generator=g, dtype=torch.int32)
        codes = torch.where((codes & 127) == 127, codes - 1, codes).to(torch.uint8)
    else:
        codes = torch.randint(-127, 128, (P, page, Hkv, D), generator=g, dtype=torch.int32).to(torch.int8)
    scales = torch.exp2(torch.randint(-12, 2, (P, page // block, Hkv), generator=g).float())
    return codes, scales


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,page,block", [(128, 8, 16, 16), (64, 3, 32, 16), (128, 1, 64, 32), (64, 5, 128, 64),
                                              (128, 2, 128, 128), (64, 1, 256, 256), (128, 3, 256, 256)])
@pytest.mark.parametrize("T", [1, 2, 17, 300])
def test_append(cuda_device, kind, D, Hkv, page, block, T):
    g = torch.Generator().manual_seed(6100 + D + Hkv + page + block + T)
    starts = [0, 1, 5, 15, 16, 31, 250, 257, 130]
    N = len(starts)
    need = [-(-(s + T) // page) for s in starts]
    P, mp = sum(need) + 3, max(need)
    perm = torch.randperm(P, generator=g)
    bt = torch.full((N, mp), -1, dtype=torch.int32)
    n = 0
    for b in range(N):
        bt[b, :need[b]] = perm[n:n + need[b]].to(torch.int32)
        n += need[b]
    kc, ks = random_pool(g, P, page, block, Hkv, D, kind)
    vc, vs = random_pool(g, P, page, block, Hkv, D, kind)
    # sizes from far below the old scales to far above them, so blocks grow and blocks stay
    size = torch.exp2(torch.randint(-14, 14, (N, T, Hkv, 1), generator=g).float())
    kn = (torch.randn(N, T, Hkv, D, generator=g) * size).to(torch.bfloat16)
    vn = (torch.randn(N, T, Hkv, D, generator=g) * 0.1).to(torch.bfloat16)
    vn[:, :, :, ::7] = 0.0
    want = orc.kv_append_q8(kc, vc, ks, vs, bt, np.array(starts), kn, vn)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    kcd, vcd, ksd, vsd, knd, vnd, btd = to(cuda_device, kc, vc, ks, vs, kn, vn, bt)
    sp = torch.tensor(starts, dtype=torch.int32, device=cuda_device)
    for _ in range(2):      # the second call with the same tokens changes nothing
        ab.kv_append_q8(knd, vnd, kcd, vcd, ksd, vsd, btd, sp, device_status=st)
        for got, ref in zip((ksd, vsd, kcd, vcd), (want[2], want[3], want[0], want[1])):
            assert np.array_equal(got.cpu().numpy(), ref.astype(got.cpu().numpy().dtype))
    assert int(st) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_append_zeros_extremes_and_not_finite(cuda_device, kind):
    g = torch.Generator().manual_seed(6200)
    kc, ks = random_pool(g, 4, 32, 16, 2, 64, kind)
    x = torch.zeros(1, 64, 2, 64, dtype=torch.bfloat16)
    x[0, 16:32] = 3.3e38
    x[0, 20:24] = -3.3895e38      # the largest bf16
    x[0, 32:48] = 1e-38
    x[0, 50, 0, 3] = float("nan")
    x[0, 51, 1, 7] = -float("inf")
    x[0, 52] = 2.0
    bt = torch.tensor([[2, 1]], dtype=torch.int32)
    sp = torch.zeros(1, dtype=torch.int32)
    want = orc.kv_append_q8(kc, kc, ks, ks, bt, np.array([0]), x, x)
    kcd, ksd, vcd, vsd, xd, btd, spd = to(cuda_device, kc, ks, kc, ks, x, bt, sp)
    ab.kv_append_q8(xd, xd, kcd, vcd, ksd, vsd, btd, spd)
    assert np.array_equal(ksd.cpu().numpy(), want[2].astype(np.float32), equal_nan=True)
    assert torch.isnan(ksd[1, 1]).all() and torch.isnan(vsd[1, 1]).all() and not torch.isnan(ksd[[0, 2, 3]]).any()
    assert np.array_equal(kcd.cpu().numpy()[[0, 2, 3]], want[0][[0, 2, 3]])
    assert np.array_equal(kcd.cpu().numpy()[1, :16], want[0][1, :16])
    # the poisoned block reads as NaN, and is sound again once written from its first slot
    k, _ = ab.kv_read_q8(kcd, vcd, ksd, vsd, btd, torch.tensor([64], dtype=torch.int32, device=cuda_device))
    assert torch.isnan(k[0, 48:]).all() and torch.isfinite(k[0, :48]).all()
    ab.kv_append_q8(xd[:, 52:53].contiguous(), xd[:, 52:53].contiguous(), kcd, vcd, ksd, vsd, btd,
                    torch.tensor([48], dtype=torch.int32, device=cuda_device))
    assert torch.isfinite(ksd).all()


def test_append_out_of_range_is_skipped_and_reported(cuda_device):
    g = torch.Generator().manual_seed(6201)
    kc, ks = random_pool(g, 4, 16, 16, 2, 128, "int8")
    x = torch.randn(4, 20, 2, 128, generator=g).to(torch.bfloat16)
    bt = torch.tensor([[0, -1], [9, 1], [2, 3], [1, 1]], dtype=torch.int32)
    starts = [3, 2, 30, -30]        # page -1; page outside; past the table; before the table
    kcd, ksd, xd, btd = to(cuda_device, kc, ks, x, bt)
    vcd, vsd = kcd.clone(), ksd.clone()
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    ab.kv_append_q8(xd, xd, kcd, vcd, ksd, vsd, btd, torch.tensor(starts, dtype=torch.int32, device=cuda_device),
                    device_status=st)
    assert int(st) == 4
    # sequence 0 wrote slots 3 .. 15 of page 0, sequence 1 slots 0 .. 5 of page 1, sequence 2 slots 14, 15 of page 3
    want = orc.kv_append_q8(kc, kc, ks, ks, bt[:1, :1], np.array([3]), x[:1, :13], x[:1, :13])
    want = orc.kv_append_q8(want[0], want[1], want[2], want[3], bt[1:2], np.array([16]), x[1:2, 14:], x[1:2, 14:])
    want = orc.kv_append_q8(want[0], want[1], want[2], want[3], bt[2:3], np.array([30]), x[2:3, :2], x[2:3, :2])
    assert np.array_equal(kcd.cpu().numpy(), want[0]) and np.array_equal(vcd.cpu().numpy(), want[1])
    assert np.array_equal(ksd.cpu().double().numpy(), want[2])


# ------------------------------------------------------------------ reading back

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,page,block", [(128, 8, 16, 16), (64, 3, 32, 32), (128, 5, 256, 64), (64, 1, 64, 16)])
def test_read_back(cuda_device, kind, D, Hkv, page, block):
    lens = [0, 1, 15, 16, 17, 300, 511]
    cache = gen.paged_decode_inputs(len(lens), Hkv, Hkv, D, page, 0, 0, seed=6300 + D + Hkv, lens=lens)
    kc, vc, ks, vs = quantized(cache, block, kind)
    k, v = orc.q8_dequant(kc, ks), orc.q8_dequant(vc, vs)
    args = to(cuda_device, kc, vc, ks, vs, cache.block_table, cache.seq_lens)
    for T in (511, 100, None):
        if T is None:
            ko, vo = ab.kv_read_q8(*args)
            fill = 0.0
        else:
            fill = 7.0
            ko = torch.full((len(lens), T, Hkv, D), fill, dtype=torch.bfloat16, device=cuda_device)
            vo = torch.full_like(ko, fill)
            ab.kv_read_q8(*args, k_out=ko, v_out=vo)
        for b, L in enumerate(lens):
            n = min(L, ko.shape[1])
            ids = cache.block_table[b, :-(-L // page)].numpy()
            for got, pool in ((ko, k), (vo, v)):
                ref = pool[ids].reshape(-1, Hkv, D)[:n]
                assert np.array_equal(got[b, :n].double().cpu().numpy(), ref)     # nothing is rounded
                assert (got[b, n:] == fill).all()


def test_read_back_foreign_scales_and_bad_pages(cuda_device):
    g = torch.Generator().manual_seed(6310)
    kc, _ = random_pool(g, 5, 16, 16, 2, 64, "int8")
    kc[0, 0, 0, 0] = -128
    ks = torch.rand(5, 1, 2, generator=g) * 3
    bt = torch.tensor([[0, 7, 3], [-1, 2, 4]], dtype=torch.int32)
    sl = torch.tensor([48, 99], dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    args = to(cuda_device, kc, kc, ks, ks, bt, sl)
    k, v = ab.kv_read_q8(*args, device_status=st)
    assert int(st) == 4
    val = (kc.float() * ks.repeat_interleave(16, dim=1)[..., None]).to(torch.bfloat16)   # one rounding
    want = torch.zeros(2, 48, 2, 64, dtype=torch.bfloat16)
    for b in range(2):
        for i in range(3):
            if 0 <= int(bt[b, i]) < 5:
                want[b, 16 * i:16 * i + 16] = val[int(bt[b, i])]
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)


# ------------------------------------------------------------------ decode

LENS = [1, 15, 16, 17, 63, 700, 2049, 0, 130]


def check_decode(dev, cache, codes, label, lens):
    kc, vc, ks, vs = codes
    scale = gen.attn_scale(cache.q.shape[-1])
    o_ref, lse_ref = orc.decode_paged_q8(cache.q, kc, vc, ks, vs, cache.block_table, cache.seq_lens, scale)
    o_ref, lse_ref = empty_rows(o_ref, lse_ref, lens)
    args = to(dev, cache.q, kc, vc, ks, vs, cache.block_table, cache.seq_lens)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    o, lse = ab.decode_paged_q8(*args, scale=scale, device_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    print(label, compare_output(o, o_ref, lse, lse_ref, label=label))
    for b, L in enumerate(lens):      # alone, the sequence is cut elsewhere
        one = [args[0][b:b + 1], *args[1:5], args[5][b:b + 1], args[6][b:b + 1]]
        o, lse = ab.decode_paged_q8(*one, scale=scale)
        compare_output(o, o_ref[b:b + 1], lse, lse_ref[b:b + 1], label=f"{label} alone {b}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D,page,block", [
    (32, 8, 128, 16, 16), (4, 4, 128, 32, 32), (1, 1, 64, 16, 16), (16, 1, 128, 64, 16), (16, 2, 64, 256, 256),
    (6, 2, 128, 16, 16), (15, 3, 64, 64, 32), (7, 1, 128, 128, 128), (27, 3, 128, 32, 16), (10, 5, 64, 16, 16),
    (44, 4, 64, 16, 16)])
def test_decode(cuda_device, kind, Hq, Hkv, D, page, block):
    cache = gen.paged_decode_inputs(len(LENS), Hq, Hkv, D, page, 0, 0, seed=6400 + Hq + Hkv + page, lens=LENS)
    codes = quantized(cache, block, kind)
    for s in codes[2:]:      # scales of blocks that hold no token
        used = torch.zeros(s.shape[:2], dtype=torch.bool)
        for b, L in enumerate(LENS):
            for t in range(0, L, block):
                used[cache.block_table[b, t // page], t % page // block] = True
        s[~used] = float("nan")
    check_decode(cuda_device, cache, codes, f"decode {kind}", LENS)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N,Hq,Hkv,D,cap", [(11, 8, 2, 128, 512), (700, 4, 2, 64, 512), (700, 4, 2, 64, 640),
                                            (333, 3, 3, 128, 160), (40, 26, 13, 128, 768), (70, 22, 22, 64, 528)])
def test_decode_many_short_sequences(cuda_device, kind, N, Hq, Hkv, D, cap):
    """Batches of many sequences (more than the 64 sums and the 32-wide window of the work walk), tables of at
    most 512 tokens (whole sequences a CTA) and of more (runs of tiles), head counts that do not divide a team."""
    g = torch.Generator().manual_seed(6450 + N + cap)
    lens = torch.randint(0, cap + 1, (N,), generator=g)
    lens[torch.randperm(N, generator=g)[:N // 5]] = 0
    lens[torch.randperm(N, generator=g)[:4]] = torch.tensor([cap, 1, 128, 129])
    lens = lens.tolist()
    cache = gen.paged_decode_inputs(N, Hq, Hkv, D, 16, 0, 0, seed=6451, lens=lens, max_pages=cap // 16, poison=False)
    codes = quantized(cache, 16, kind)
    scale = gen.attn_scale(D)
    o_ref, lse_ref = orc.decode_paged_q8(cache.q, *codes[:2], *codes[2:], cache.block_table, cache.seq_lens, scale)
    o_ref, lse_ref = empty_rows(o_ref, lse_ref, lens)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    o, lse = ab.decode_paged_q8(*to(cuda_device, cache.q, *codes, cache.block_table, cache.seq_lens), scale=scale,
                                device_status=st)
    assert int(st) == 0
    compare_output(o, o_ref, lse, lse_ref, label=f"{kind} N={N}")


@pytest.mark.parametrize("kind", KINDS)
def test_decode_full_size(cuda_device, kind):
    """64 sequences, lengths uniform in [512, 8192], Hq=32, Hkv=8, D=128, page 16, one scale per 16 tokens."""
    c = gen.CONFIGS["paged_gqa_decode"]
    cache = gen.paged_decode_inputs(c["N"], c["Hq"], c["Hkv"], c["D"], c["page_size"], c["len_lo"], c["len_hi"],
                                    seed=c["seed"])
    check_decode(cuda_device, cache, quantized(cache, 16, kind), f"decode full {kind}", cache.seq_lens)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 128), (8, 2, 64), (16, 2, 128), (32, 2, 128), (32, 4, 64), (32, 2, 64)])
def test_decode_lse_keeps_fp32(cuda_device, kind, Hq, Hkv, D):
    """One token: the LSE is its score alone. q's digits are off by 2^-22 of the row's largest value (|q| < 6),
    the products are exact in int32; E4M3 products are summed in fp32, 128 terms of at most |q k| scale < 6 * 5 *
    0.125 that may each round by 2^-24 of the sum's size (< 16). So |error| < 128 * (6 * 2^-22 * 5 * 0.125 + 2^-24 *
    16) = 2.4e-4 if all went one way; independent ones add up to 1 / sqrt(128) of it, 2.1e-5, and typical values
    (|q|, |k| = 1, a few elements of q below 2^-14 of the largest, sums of size 1) to less than a tenth of that.
    (Two int8 digits alone give an rms of 4e-6 and a maximum of 2.6e-5.)"""
    lens = [1] * 64
    cache = gen.paged_decode_inputs(64, Hq, Hkv, D, 16, 0, 0, seed=6470 + Hq + D, lens=lens, poison=False)
    codes = quantized(cache, 16, kind)
    scale = gen.attn_scale(D)
    o_ref, lse_ref = orc.decode_paged_q8(cache.q, *codes, cache.block_table, cache.seq_lens, scale)
    o, lse = ab.decode_paged_q8(*to(cuda_device, cache.q, *codes, cache.block_table, cache.seq_lens), scale=scale)
    err = lse.cpu().numpy() - lse_ref
    print(kind, "max", np.abs(err).max(), "rms", np.sqrt((err ** 2).mean()))
    assert np.sqrt((err ** 2).mean()) < 2.1e-6 and np.abs(err).max() < 2.1e-5


@pytest.mark.parametrize("kind", KINDS)
def test_decode_dominant_key(cuda_device, kind):
    S = 3000
    q, k, v = gen.peaked_prefill_inputs(1, 32, 8, S, 128, seed=6500, amp=12.0, period=S)
    cache = gen.paged_from_contiguous(q[:, S - 1], k, v, page_size=16, seed=6501)
    check_decode(cuda_device, cache, quantized(cache, 16, kind), f"dominant {kind}", [S])


@pytest.mark.parametrize("kind", KINDS)
def test_decode_value_scales_far_apart(cuda_device, kind):
    """V scales from 2^-60 to 2^40 by block, K scales from 2^-12 to 2^2: the value scale is part of the
    exponent, so no block's share is lost. Each output is off by the digits' rounding of the weights, at most
    2^-9 of sum |P V|, the products' fp32 sums and exponentials (2^-20 of it for the 2^4 log2 units here), and
    half a bf16 step."""
    g = torch.Generator().manual_seed(6510)
    lens = [1, 40, 333, 1000]
    cache = gen.paged_decode_inputs(len(lens), 8, 2, 128, 32, 0, 0, seed=6511, lens=lens, poison=False)
    kc, vc, ks, vs = quantized(cache, 16, kind)
    vs = torch.exp2(torch.randint(-60, 41, vs.shape, generator=g).float())
    ks = ks * torch.exp2(torch.randint(-8, 1, ks.shape, generator=g).float())
    scale = gen.attn_scale(128)
    o_ref, lse_ref = orc.decode_paged_q8(cache.q, kc, vc, ks, vs, cache.block_table, cache.seq_lens, scale)
    absv = np.abs(orc.q8_dequant(vc, vs))
    bound, _ = orc.decode_paged(cache.q, orc.q8_dequant(kc, ks), absv, cache.block_table, cache.seq_lens, 32, scale)
    args = to(cuda_device, cache.q, kc, vc, ks, vs, cache.block_table, cache.seq_lens)
    o, lse = ab.decode_paged_q8(*args, scale=scale)
    err = np.abs(o.double().cpu().numpy() - o_ref)
    assert (err <= (2.0 ** -9 + 2.0 ** -16) * bound + 2.0 ** -9 * np.abs(o_ref) * 1.01).all()
    assert np.abs(lse.double().cpu().numpy() - lse_ref).max() <= 1e-3


@pytest.mark.parametrize("kind", KINDS)
def test_decode_zero_scales_and_foreign_ones(cuda_device, kind):
    g = torch.Generator().manual_seed(6520)
    lens = [5, 64, 200]
    cache = gen.paged_decode_inputs(len(lens), 4, 2, 64, 16, 0, 0, seed=6521, lens=lens, poison=False)
    kc, vc, ks, vs = quantized(cache, 16, kind)
    ks, vs = torch.rand(ks.shape, generator=g) * 0.02, torch.rand(vs.shape, generator=g) * 0.02
    ks[::3], vs[::2] = 0.0, 0.0
    check_decode(cuda_device, cache, (kc, vc, ks, vs), f"foreign scales {kind}", lens)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_nan_stays_with_its_rows(cuda_device, kind):
    """A NaN K scale, a NaN V scale and queries that are not finite poison the outputs that see them, and
    no others."""
    lens = [100, 100, 600, 600, 40]
    cache = gen.paged_decode_inputs(len(lens), 8, 2, 64, 16, 0, 0, seed=6530, lens=lens, poison=False)
    kc, vc, ks, vs = quantized(cache, 16, kind)
    scale = gen.attn_scale(64)
    o_ref, _ = orc.decode_paged_q8(cache.q, kc, vc, ks, vs, cache.block_table, cache.seq_lens, scale)
    q = cache.q.clone()
    ks[cache.block_table[0, 3].long(), 0, 1] = float("nan")
    vs[cache.block_table[2, 20].long(), 0, 0] = float("nan")
    q[3, 5, 9] = float("inf")
    q[4, 0, 0] = float("nan")
    o, lse = ab.decode_paged_q8(*to(cuda_device, q, kc, vc, ks, vs, cache.block_table, cache.seq_lens), scale=scale)
    o, lse = o.float().cpu().numpy(), lse.cpu().numpy()
    bad = np.zeros((5, 8), bool)
    bad[0, 4:], bad[2, :4], bad[3, 5], bad[4, 0] = True, True, True, True
    assert np.isnan(o[bad]).all()
    assert np.isfinite(lse[~bad]).all()
    compare_output(o, np.where(bad[..., None], 0.0, o_ref), mask=~np.repeat(bad[..., None], 64, -1))


def test_decode_bad_pages_and_lengths(cuda_device):
    cache = gen.paged_decode_inputs(4, 8, 2, 128, 16, 0, 0, seed=6540, lens=[100, 200, 64, 64], max_pages=13)
    kc, vc, ks, vs = quantized(cache, 16, "e4m3")
    scale = gen.attn_scale(128)
    bt = cache.block_table.clone()
    bt[0, 2], bt[1, 12], bt[2] = -1, 10 ** 6, -5
    sl = cache.seq_lens.clone()
    sl[1], sl[3] = 500, -3            # beyond the table's 208 slots; negative
    bt[1, 12] = 10 ** 6
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    o, lse = ab.decode_paged_q8(*to(cuda_device, cache.q, kc, vc, ks, vs, bt, sl), scale=scale, device_status=st)
    assert int(st) == 4
    k, v = orc.q8_dequant(kc, ks), orc.q8_dequant(vc, vs)
    for b, L in ((0, 100), (1, 208)):
        toks = [t for t in range(L) if 0 <= int(bt[b, t // 16]) < k.shape[0]]
        toks = [t for t in toks if t < int(cache.seq_lens[b]) or b == 0]
        kk = np.stack([k[int(bt[b, t // 16]), t % 16] for t in toks])
        vv = np.stack([v[int(bt[b, t // 16]), t % 16] for t in toks])
        if b == 1:                    # slots 192 .. 207 sit on the page outside the pool, the rest is held
            assert len(toks) == 192
        table, n = torch.arange(-(-len(toks) // 16), dtype=torch.int32)[None], len(toks)
        pad = -n % 16
        pk = np.concatenate([kk, np.zeros((pad,) + kk.shape[1:])]).reshape(-1, 16, 2, 128)
        pv = np.concatenate([vv, np.zeros((pad,) + vv.shape[1:])]).reshape(-1, 16, 2, 128)
        o_ref, l_ref = orc.decode_paged(cache.q[b:b + 1], pk, pv, table, torch.tensor([n]), 16, scale)
        compare_output(o[b:b + 1], o_ref, lse[b:b + 1], l_ref, label=f"sequence {b}")
    assert (o[2:] == 0).all() and torch.isneginf(lse[2:]).all()


def test_decode_nan_codes_stay_with_their_head(cuda_device):
    """Two heads of D = 64 share a 128-byte row of a tile: an E4M3 NaN code of one head's key or value must not
    reach the other's outputs."""
    lens = [200, 90, 300]
    cache = gen.paged_decode_inputs(len(lens), 8, 4, 64, 16, 0, 0, seed=6550, lens=lens, poison=False)
    kc, vc, ks, vs = quantized(cache, 16, "e4m3")
    scale = gen.attn_scale(64)
    o_ref, lse_ref = orc.decode_paged_q8(cache.q, kc, vc, ks, vs, cache.block_table, cache.seq_lens, scale)
    kc[cache.block_table[0, 3].long(), 5, 1, 7] = 0x7F        # a key of head 1
    vc[cache.block_table[2, 2].long(), 9, 2, 11] = 0xFF       # one dimension of a value of head 2
    o, lse = ab.decode_paged_q8(*to(cuda_device, cache.q, kc, vc, ks, vs, cache.block_table, cache.seq_lens), scale=scale)
    o = o.float().cpu().numpy()
    bad = np.zeros(o.shape, bool)
    bad[0, 2:4] = True
    bad[2, 4:6, 11] = True
    assert np.isnan(o[bad]).all()
    compare_output(o, np.where(bad, 0.0, o_ref), mask=~bad)
    ok = ~bad.all(-1)
    assert np.abs(lse.cpu().numpy()[ok] - lse_ref[ok]).max() <= 1e-3


@pytest.mark.parametrize("kind", KINDS)
def test_pages_beyond_four_gigabytes(cuda_device, kind):
    """Append, read back and decode on pages whose codes lie past 2^32 bytes of the pool."""
    g = torch.Generator().manual_seed(6560)
    page, block, Hkv, D, T = 256, 32, 8, 128, 300
    P = 17000                                             # 4.46e9 codes in each pool
    dt = torch.uint8 if kind == "e4m3" else torch.int8
    kc = torch.zeros(P, page, Hkv, D, dtype=dt, device=cuda_device)
    vc = torch.zeros_like(kc)
    ks = torch.ones(P, page // block, Hkv, device=cuda_device)
    vs = torch.ones_like(ks)
    bt = torch.tensor([[P - 1, P - 3], [16500, 2]], dtype=torch.int32, device=cuda_device)
    kn, vn = [torch.randn(2, T, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2)]
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    ab.kv_append_q8(*to(cuda_device, kn, vn), kc, vc, ks, vs, bt, torch.zeros(2, dtype=torch.int32, device=cuda_device),
                    device_status=st)
    # the oracle sees the four pages alone
    ids = bt.flatten().long()
    small = torch.arange(4, dtype=torch.int32).view(2, 2)
    z = np.zeros((4, page, Hkv, D), np.uint8 if kind == "e4m3" else np.int8)
    one = np.ones((4, page // block, Hkv))
    ref = orc.kv_append_q8(z, z, one, one, small, np.zeros(2, int), kn, vn)
    for got, want in zip((kc, vc, ks, vs), ref):
        assert np.array_equal(got[ids].cpu().numpy(), want.astype(got[ids].cpu().numpy().dtype))
    sl = torch.tensor([T, T], dtype=torch.int32, device=cuda_device)
    k, v = ab.kv_read_q8(kc, vc, ks, vs, bt, sl, num_tokens=T, device_status=st)
    pool = orc.q8_dequant(ref[0], ref[2]).reshape(2, 2 * page, Hkv, D)[:, :T]
    assert np.array_equal(k.double().cpu().numpy(), pool)
    q = torch.randn(2, 32, D, generator=g).to(torch.bfloat16)
    o, lse = ab.decode_paged_q8(q.to(cuda_device), kc, vc, ks, vs, bt, sl, device_status=st)
    o_ref, l_ref = orc.decode_paged_q8(q, *ref, small, sl.cpu(), gen.attn_scale(D))
    compare_output(o, o_ref, lse, l_ref, label=f"far pages {kind}")
    assert int(st) == 0


# ------------------------------------------------------------------ prefill, and the loop of them

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D,page,block,Sq", [(8, 2, 128, 16, 16, 100), (6, 2, 64, 64, 32, 257),
                                                    (4, 4, 128, 256, 256, 1), (12, 1, 64, 32, 16, 33)])
def test_prefill(cuda_device, kind, Hq, Hkv, D, page, block, Sq):
    lens = [Sq, Sq + 1, Sq + 200, 500]
    c = gen.paged_prefill_inputs(4, Sq, Hq, Hkv, D, page, lens, seed=6600 + Hq + D)
    kc, vc, ks, vs = quantized(c, block, kind)
    scale = gen.attn_scale(D)
    o_ref, lse_ref = orc.prefill_paged_q8(c.q, kc, vc, ks, vs, c.block_table, c.seq_lens, scale)
    args = to(cuda_device, c.q, kc, vc, ks, vs, c.block_table, c.seq_lens)
    ws = torch.full((ab.binding.prefill_paged_q8_workspace_bytes(4, Hkv, D, c.block_table.shape[1], page),), 255,
                    dtype=torch.uint8, device=cuda_device)          # NaN in every scratch slot
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    o, lse = ab.prefill_paged_q8(*args, scale=scale, workspace=ws, device_status=st)
    assert int(st) == 0
    compare_output(o, o_ref, lse, lse_ref, label=f"prefill {kind}")
    o2, lse2 = ab.prefill_paged_q8(*args, scale=scale)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_nan_reaches_only_the_queries_that_see_it(cuda_device, kind):
    """NaN scales (and E4M3 NaN codes) of keys and values inside the chunk, hidden from its earlier queries by
    the causal mask but in their key tiles: those queries are untouched, the later ones NaN."""
    Sq, lens, block = 120, [120, 300, 250, 131], 16
    c = gen.paged_prefill_inputs(4, Sq, 4, 2, 128, 16, lens, seed=6640, poison=False)
    kc, vc, ks, vs = quantized(c, block, kind)
    scale = gen.attn_scale(128)
    o_ref, lse_ref = orc.prefill_paged_q8(c.q, kc, vc, ks, vs, c.block_table, c.seq_lens, scale)
    page = lambda b, t: int(c.block_table[b, t // 16])
    seen_from = [None] * 4                    # (first position that sees it, KV head)
    vs[page(0, 64), 0, 0] = float("nan")
    seen_from[0] = (64, 0)
    ks[page(1, 240), 0, 1] = float("nan")
    seen_from[1] = (240, 1)
    if kind == "e4m3":
        vc[page(2, 203), 203 % 16, 1, 100] = 0x7F
        seen_from[2] = (203, 1)
        kc[page(3, 130), 130 % 16, 0, 3] = 0xFF
        seen_from[3] = (130, 0)
    o, lse = ab.prefill_paged_q8(*to(cuda_device, c.q, kc, vc, ks, vs, c.block_table, c.seq_lens), scale=scale)
    bad = np.zeros(o.shape, bool)             # [B, Sq, Hq, D]
    for b, at in enumerate(seen_from):
        if at is not None:
            bad[b, at[0] - (lens[b] - Sq):, at[1] * 2:at[1] * 2 + 2] = True
    o, lse = o.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isnan(o[bad]).all()
    compare_output(o, np.where(bad, 0.0, o_ref), mask=~bad)
    row_bad = bad.any(-1).transpose(0, 2, 1)
    assert np.isnan(lse[row_bad]).all()
    assert np.abs(lse[~row_bad] - lse_ref[~row_bad]).max() <= 1e-3


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D,Sq,lens,pages", [
    (4, 1, 128, 1, [4000, 1, 700], 256), (2, 2, 64, 130, [130, 3100, 257, 1500], 200),
    (16, 4, 64, 117, [117, 2400, 1300], 150), (1, 1, 128, 300, [6000], 375), (3, 3, 128, 200, [700], 44),
    (8, 2, 64, 513, [513, 2047], 128), (70, 10, 64, 7, [1111], 70)])
def test_prefill_few_items(cuda_device, kind, Hq, Hkv, D, Sq, lens, pages):
    """Short chunks after long prefixes on few heads: the key tiles of an item are cut over several CTAs, some
    sequences of the batch having fewer tiles than there are parts."""
    c = gen.paged_prefill_inputs(len(lens), Sq, Hq, Hkv, D, 16, lens, seed=6630 + Hq + Sq)
    kc, vc, ks, vs = quantized(c, 16, kind)
    bt = torch.full((len(lens), pages), -1, dtype=torch.int32)
    bt[:, :c.block_table.shape[1]] = c.block_table
    scale = gen.attn_scale(D)
    o_ref, lse_ref = orc.prefill_paged_q8(c.q, kc, vc, ks, vs, bt, c.seq_lens, scale)
    args = to(cuda_device, c.q, kc, vc, ks, vs, bt, c.seq_lens)
    ws = torch.full((ab.binding.prefill_paged_q8_workspace_bytes(len(lens), Hkv, D, pages, 16),), 255,
                    dtype=torch.uint8, device=cuda_device)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    o, lse = ab.prefill_paged_q8(*args, scale=scale, workspace=ws, device_status=st)
    assert int(st) == 0
    compare_output(o, o_ref, lse, lse_ref, label=f"few items {kind}")
    o2, none = ab.prefill_paged_q8(*args, scale=scale, return_lse=False)
    assert torch.equal(o, o2) and none is None


def test_prefill_bad_pages_and_lengths(cuda_device):
    """As the bf16 chunked prefill: keys of a page outside the pool read as zeros, a length outside
    [Sq, capacity] is clamped, both reported; the other sequences are untouched."""
    Sq, lens = 40, [100, 90, 64]
    c = gen.paged_prefill_inputs(3, Sq, 4, 2, 64, 16, lens, seed=6650, poison=False)
    kc, vc, ks, vs = quantized(c, 16, "int8")
    scale = gen.attn_scale(64)
    bt, sl = c.block_table.clone(), c.seq_lens.clone()
    bad_page = int(bt[0, 1])
    bt[0, 1] = 10 ** 7
    sl[1] = 10 ** 6                       # clamped to the table's capacity: 112 tokens
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    o, lse = ab.prefill_paged_q8(*to(cuda_device, c.q, kc, vc, ks, vs, bt, sl), scale=scale, device_status=st)
    assert int(st) == 4
    zk, zv = kc.clone(), vc.clone()
    zk[bad_page], zv[bad_page] = 0, 0
    o_ref, l_ref = orc.prefill_paged_q8(c.q, zk, zv, ks, vs, c.block_table, c.seq_lens, scale, seqs=[0, 2])
    for b in (0, 2):
        compare_output(o[b], o_ref[b], lse[b], l_ref[b], label=f"sequence {b}")
    o1, _ = ab.prefill_paged_q8(*to(cuda_device, c.q[2:].contiguous(), kc, vc, ks, vs, bt[2:], sl[2:]), scale=scale)
    assert torch.equal(o1[0], o[2])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hq,Hkv,page,block", [(128, 8, 2, 16, 16), (64, 6, 3, 64, 32)])
def test_serving_loop(cuda_device, kind, D, Hq, Hkv, page, block):
    """Prompts in two chunks (append, prefill), then tokens one by one (append, decode): every attention
    output against the oracle on the codes the loop itself has written, the codes against the oracle's."""
    g = torch.Generator().manual_seed(6700)
    N, chunks, steps = 3, (40, 25), 6
    total = sum(chunks) + steps
    mp = -(-(total + 7) // page)
    P = N * mp + 2
    bt = torch.randperm(P, generator=g)[:N * mp].view(N, mp).to(torch.int32)
    dt = np.uint8 if kind == "e4m3" else np.int8
    ref = [np.zeros((P, page, Hkv, D), dt) for _ in range(2)] + [np.zeros((P, page // block, Hkv)) for _ in range(2)]
    kc, vc = [torch.tensor(x, device=cuda_device) for x in ref[:2]]
    ks, vs = [torch.tensor(x, dtype=torch.float32, device=cuda_device) for x in ref[2:]]
    btd = bt.to(cuda_device)
    lens = torch.tensor([0, 3, 7], dtype=torch.int32)      # some sequences start behind a few tokens
    first = (0.3 * torch.randn(N, 7, Hkv, D, generator=g)).to(torch.bfloat16)
    for b in range(N):
        if int(lens[b]):
            n = int(lens[b])
            ab.kv_append_q8(*to(cuda_device, first[b:b + 1, :n].contiguous(), first[b:b + 1, :n].contiguous()), kc, vc, ks,
                            vs, btd[b:b + 1], torch.zeros(1, dtype=torch.int32, device=cuda_device))
            ref = list(orc.kv_append_q8(*ref, bt[b:b + 1], np.array([0]), first[b:b + 1, :n], first[b:b + 1, :n]))
    scale = gen.attn_scale(D)
    for i, T in enumerate(list(chunks) + [1] * steps):
        size = 1.0 + 0.5 * i                                 # later tokens are larger: scales grow
        kn = (size * torch.randn(N, T, Hkv, D, generator=g)).to(torch.bfloat16)
        vn = (size * torch.randn(N, T, Hkv, D, generator=g)).to(torch.bfloat16)
        ab.kv_append_q8(*to(cuda_device, kn, vn), kc, vc, ks, vs, btd, lens.to(cuda_device))
        ref = list(orc.kv_append_q8(*ref, bt, lens.numpy(), kn, vn))
        lens = lens + T
        for got, want in zip((kc, vc, ks, vs), ref):
            assert np.array_equal(got.cpu().numpy(), want.astype(got.cpu().numpy().dtype))
        q = torch.randn(N, T, Hq, D, generator=g).to(torch.bfloat16)
        ld = lens.to(cuda_device)
        if T > 1:
            o, lse = ab.prefill_paged_q8(q.to(cuda_device), kc, vc, ks, vs, btd, ld, scale=scale)
            o_ref, l_ref = orc.prefill_paged_q8(q, *ref, bt, lens, scale)
        else:
            o, lse = ab.decode_paged_q8(q[:, 0].contiguous().to(cuda_device), kc, vc, ks, vs, btd, ld, scale=scale)
            o_ref, l_ref = orc.decode_paged_q8(q[:, 0], *ref, bt, lens, scale)
        compare_output(o, o_ref, lse, l_ref, label=f"step {i}")


@pytest.mark.parametrize("kind", KINDS)
def test_graph_stream_and_repeats(cuda_device, kind):
    """Captured and replayed on another stream, the calls give the eager results bit for bit, after the
    inputs change too; so do repeated eager calls."""
    g = torch.Generator().manual_seed(6800)
    lens = [300, 1000, 1, 77]
    cache = gen.paged_decode_inputs(4, 16, 4, 128, 32, 0, 0, seed=6801, lens=lens, poison=False, max_pages=40)
    kc, vc, ks, vs = to(cuda_device, *quantized(cache, 16, kind))
    q, bt, sl = to(cuda_device, cache.q, cache.block_table, cache.seq_lens)
    sp = sl - 1
    kn = torch.randn(4, 1, 4, 128, generator=g).to(torch.bfloat16).to(cuda_device)
    qp = torch.randn(4, 1, 16, 128, generator=g).to(torch.bfloat16).to(cuda_device)

    def step():
        ab.kv_append_q8(kn, kn, kc, vc, ks, vs, bt, sp)
        o, lse = ab.decode_paged_q8(q, kc, vc, ks, vs, bt, sl)
        op, lp = ab.prefill_paged_q8(qp, kc, vc, ks, vs, bt, sl)
        k, v = ab.kv_read_q8(kc, vc, ks, vs, bt, sl)
        return o, lse, op, lp, k, v

    want = [t.clone() for t in step()]
    for got, ref in zip(step(), want):
        assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream(device=cuda_device)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        outs = step()
    graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        assert torch.equal(got, ref)
    q.copy_(torch.randn(q.shape, generator=g).to(torch.bfloat16))
    kn.mul_(3)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in outs]
    again = torch.cuda.Stream(device=cuda_device)
    again.wait_stream(torch.cuda.current_stream())
    o, lse = ab.decode_paged_q8(q, kc, vc, ks, vs, bt, sl, stream=again)   # outputs belong to that stream
    again.synchronize()
    assert torch.equal(o, got[0]) and torch.equal(lse, got[1]) and not torch.equal(o, want[0])


def test_cut_prefill_in_a_graph_and_on_two_streams(cuda_device):
    """The prefill whose key tiles are cut (three dependent launches): captured twice into one graph with one
    workspace, replayed on new queries, and two calls at once on two streams."""
    c = gen.paged_prefill_inputs(2, 90, 4, 2, 128, 16, [3000, 1200], seed=6830, poison=False)
    kc, vc, ks, vs = to(cuda_device, *quantized(c, 16, "int8"))
    q, bt, sl = to(cuda_device, c.q, c.block_table, c.seq_lens)
    ws = torch.empty(ab.binding.prefill_paged_q8_workspace_bytes(2, 2, 128, bt.shape[1], 16), dtype=torch.uint8,
                     device=cuda_device)
    q2 = q.flip(0).contiguous()
    step = lambda: (*ab.prefill_paged_q8(q, kc, vc, ks, vs, bt, sl, workspace=ws),
                    *ab.prefill_paged_q8(q2, kc, vc, ks, vs, bt, sl, workspace=ws))
    want = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for t in (q, q2):
        t.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    half = [t.clone() for t in step()]
    for a, b, w in zip(outs, half, want):
        assert torch.equal(a, b) and not torch.equal(a, w)
    streams = [torch.cuda.Stream(device=cuda_device) for _ in range(2)]
    torch.cuda.synchronize()
    rows = [[ab.prefill_paged_q8(x, kc, vc, ks, vs, bt, sl, stream=s) for x, s in zip((q, q2), streams)]
            for _ in range(5)]
    torch.cuda.synchronize()
    for (o, l), (o2, l2) in rows:
        assert torch.equal(o, half[0]) and torch.equal(l, half[1])
        assert torch.equal(o2, half[2]) and torch.equal(l2, half[3])


def test_two_streams_at_once(cuda_device):
    lens = [2000, 1500, 900, 40]
    cache = gen.paged_decode_inputs(4, 16, 4, 128, 16, 0, 0, seed=6810, lens=lens, poison=False)
    args = to(cuda_device, cache.q, *quantized(cache, 16, "int8"), cache.block_table, cache.seq_lens)
    want, wl = ab.decode_paged_q8(*args)
    streams = [torch.cuda.Stream(device=cuda_device) for _ in range(3)]
    torch.cuda.synchronize()
    outs = [[ab.decode_paged_q8(*args, stream=s) for s in streams] for _ in range(5)]
    torch.cuda.synchronize()
    for row in outs:
        for o, lse in row:
            assert torch.equal(o, want) and torch.equal(lse, wl)


def test_binding_refusals(cuda_device):
    cache = gen.paged_decode_inputs(2, 4, 2, 64, 32, 0, 0, seed=6900, lens=[5, 40], poison=False)
    kc, vc, ks, vs = to(cuda_device, *quantized(cache, 16, "e4m3"))
    q, bt, sl = to(cuda_device, cache.q, cache.block_table, cache.seq_lens)
    good = dict(q=q, k_codes=kc, v_codes=vc, k_scales=ks, v_scales=vs, block_table=bt, seq_lens=sl)
    ab.decode_paged_q8(**good)
    for bad in (dict(v_codes=vc.view(torch.int8)), dict(v_scales=vs[:, :1].contiguous()), dict(k_scales=ks.double()),
                dict(seq_lens=sl[:1]), dict(q=q[:1]), dict(q=q.float()), dict(q=q.transpose(0, 1)),
                dict(k_codes=kc[:, ::2]), dict(block_table=bt.cpu()), dict(out=torch.empty_like(q)[:, :2]),
                dict(lse=torch.empty(2, 5, device=cuda_device)),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device=cuda_device)),
                dict(device_status=torch.zeros(1, device=cuda_device))):
        with pytest.raises(ab.AttnError):
            ab.decode_paged_q8(**(good | bad))
    with pytest.raises(ab.AttnError):
        ab.kv_read_q8(kc, vc, ks, vs, bt, sl, num_tokens=bt.shape[1] * 32 + 1)
    with pytest.raises(ab.AttnError):
        ab.kv_append_q8(q[:, None], q[:, None], kc, vc, ks, vs, bt, sl)          # 4 heads into a cache of 2
