"""The 8-bit cache at the ends of its range, against 64 bits."""

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


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 128), (8, 2, 128), (32, 2, 128), (8, 4, 64), (32, 2, 64)])
@pytest.mark.parametrize("exponent", [-130, -100, 60, 104, 112, "most"])
def test_decode_value_scales_at_the_ends(cuda_device, kind, Hq, Hkv, D, exponent):
    """V scales up to the largest that the append writes: one token, several tiles, and sequences that are cut
    and merged. Every output is a weighted mean of finite values, so it is finite. Each is off by the
    weights' digits, at most 2^-9 of A = sum P |V| and 128 * 2^-22 of the largest |V|, by fp32 roundings (2^-14 A
    covers them) and by half a bf16 step, 2^-8 (below the normal range, 2^-134)."""
    top = {"e4m3": 119, "int8": 121}[kind] if exponent == "most" else exponent
    lens = [1, 2, 130, 600, 5000]
    c = gen.paged_decode_inputs(len(lens), Hq, Hkv, D, 16, 0, 0, seed=7300 + Hq + D, lens=lens, poison=False)
    kc, ks = gen.quantize_pool_q8(c.k_pages, 16, kind)
    vc, vs = gen.quantize_pool_q8(c.v_pages.abs(), 16, kind)     # one sign: sums grow
    vc = vc.clone()
    vc[c.block_table[0, 0].long(), 0] = 0x7E if kind == "e4m3" else 127     # the first sequence's one token: Q
    vs = torch.full_like(vs, 2.0 ** top)
    scale = gen.attn_scale(D)
    o_ref, l_ref = orc.decode_paged_q8(c.q, kc, vc, ks, vs, c.block_table, c.seq_lens, scale)
    a, _ = orc.decode_paged(c.q, orc.q8_dequant(kc, ks), np.abs(orc.q8_dequant(vc, vs)), c.block_table, c.seq_lens, 16,
                            scale)
    o, lse = ab.decode_paged_q8(*to(cuda_device, c.q, kc, vc, ks, vs, c.block_table, c.seq_lens), scale=scale)
    o = o.double().cpu().numpy()
    assert np.isfinite(o).all()
    largest = np.abs(orc.q8_values(vc)).max() * 2.0 ** top
    bound = 2.0 ** -8 * np.abs(o_ref) + (2.0 ** -9 + 2.0 ** -14) * a + 2.0 ** -15 * largest + 2.0 ** -134
    assert (np.abs(o - o_ref) <= bound).all()
    assert np.abs(lse.double().cpu().numpy() - l_ref).max() <= 1e-3


@pytest.mark.parametrize("D,Hq,Hkv,Sq,pages", [(128, 4, 2, 120, 20), (64, 4, 2, 120, 20), (128, 2, 2, 40, 200)])
def test_prefill_key_that_reads_as_infinity(cuda_device, D, Hq, Hkv, Sq, pages):
    """A finite scale times a code can pass the largest number: the key reads as infinity, its score is -inf for
    one sign of q and +inf for the other. The queries that see it are NaN, all of them, and no others."""
    lens = [Sq + 130, Sq]
    c = gen.paged_prefill_inputs(2, Sq, Hq, Hkv, D, 16, lens, seed=7400 + D, poison=False)
    kc, ks = gen.quantize_pool_q8(c.k_pages, 16, "e4m3")
    vc, vs = gen.quantize_pool_q8(c.v_pages, 16, "e4m3")
    bt = torch.full((2, pages), -1, dtype=torch.int32)
    bt[:, :c.block_table.shape[1]] = c.block_table
    scale = gen.attn_scale(D)
    at, head = 140, 1                           # token of sequence 0; its block holds no other key that is not zero
    page = int(bt[0, at // 16])
    kc[page, :, head] = 0
    kc[page, at % 16, head, 3] = 0x7E           # 448
    ks[page, 0, head] = 1e37
    q = c.q.clone()
    q[:, :, :, 3] = torch.where(torch.arange(Sq)[None, :, None] % 2 == 0, 1.0, -1.0).to(torch.bfloat16)
    zk = orc.q8_dequant(kc, ks)
    zk[page, :, head] = 0.0
    o_ref, l_ref = orc.prefill_paged(q, zk, orc.q8_dequant(vc, vs), bt, c.seq_lens, 16, scale)
    o, lse = ab.prefill_paged_q8(*to(cuda_device, q, kc, vc, ks, vs, bt, c.seq_lens), scale=scale)
    o, lse = o.float().cpu().numpy(), lse.cpu().numpy()
    bad = np.zeros((2, Sq, Hq), bool)
    G = Hq // Hkv
    bad[0, max(0, at - (lens[0] - Sq)):, head * G:(head + 1) * G] = True
    assert np.isnan(o[bad]).all() and np.isnan(lse.transpose(0, 2, 1)[bad]).all()
    compare_output(o, np.where(bad[..., None], 0.0, o_ref), mask=np.repeat(~bad[..., None], D, -1))
    assert np.abs(lse - l_ref)[~bad.transpose(0, 2, 1)].max() <= 1e-3


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,page,block", [(128, 2, 16, 16), (64, 3, 64, 32), (128, 1, 256, 256)])
def test_append_to_blocks_with_foreign_scales(cuda_device, kind, D, Hkv, page, block):
    """Blocks begun by another writer, with scales that are no powers of two: new codes are x / s rounded once,
    ties to even, and earlier codes c s / s' rounded once. Equal to the oracle code for code."""
    g = torch.Generator().manual_seed(7500 + D + block)
    N, T = 6, 7
    P = N + 1
    qmax = 448.0 if kind == "e4m3" else 127.0
    if kind == "e4m3":
        kc = torch.randint(0, 256, (P, page, Hkv, D), generator=g, dtype=torch.int32)
        kc = torch.where((kc & 127) == 127, kc - 1, kc).to(torch.uint8)
    else:
        kc = torch.randint(-128, 128, (P, page, Hkv, D), generator=g, dtype=torch.int32).to(torch.int8)
    vc = kc.flip(0).contiguous()
    odd = torch.tensor([3.0, 5.0, 7.0, 11.0, 1.0 / 3.0, 0.3])
    ks = odd[torch.randint(0, 6, (P, page // block, Hkv), generator=g)] * 2.0 ** -8
    vs = torch.rand(P, page // block, Hkv, generator=g) * 0.01 + 1e-4
    ks[5], vs[5] = 2e38, 3.3e38                          # the reciprocals are not normal numbers
    bt = torch.randperm(N, generator=g).to(torch.int32)[:, None]
    starts = np.array([3, 1, 9, 5, 2, 8])
    # K: halves of small multiples of the scales (ties), below the block's scale; V: some blocks grow, some stay
    page_of = bt[:, 0].long()
    n = torch.randint(0, 21, (N, T, Hkv, D), generator=g) * 2 + 1
    base = torch.tensor([3.0, 5.0, 7.0, 11.0])[torch.randint(0, 4, (N, T, Hkv, D), generator=g)]
    kn = (n * base * 2.0 ** -9 * torch.where(torch.rand(n.shape, generator=g) < 0.5, 1, -1)).to(torch.bfloat16)
    vn = (torch.randn(N, T, Hkv, D, generator=g) * torch.exp2(torch.randint(-6, 6, (N, 1, Hkv, 1), generator=g).float())
          ).to(torch.bfloat16)
    kn[page_of == 5] = 1e38
    vn[page_of == 5] = -2e38
    want = orc.kv_append_q8(kc, vc, ks, vs, bt, starts, kn, vn)
    kcd, vcd, ksd, vsd, knd, vnd, btd = to(cuda_device, kc, vc, ks, vs, kn, vn, bt)
    ab.kv_append_q8(knd, vnd, kcd, vcd, ksd, vsd, btd, torch.tensor(starts, dtype=torch.int32, device=cuda_device))
    before = ks[page_of, 0].double().numpy()
    assert (want[2][page_of.numpy(), 0] == before).any()                         # some foreign scales are kept
    for got, ref in zip((ksd, vsd, kcd, vcd), (want[2], want[3], want[0], want[1])):
        diff = got.cpu().numpy() != ref.astype(got.cpu().numpy().dtype)
        assert not diff.any(), f"{int(diff.sum())} of {diff.size} differ"


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_row_without_a_finite_score(cuda_device, D):
    """A query whose only scores pass the largest number downwards: o = 0 and an LSE of -inf, whether or not the
    table is wide enough for the keys to be cut over several CTAs."""
    kc = torch.full((2, 16, 1, D), 0x7E, dtype=torch.uint8)          # 448 * 2^119, a finite bf16
    vc = torch.full((2, 16, 1, D), 0x38, dtype=torch.uint8)          # 1
    ks, vs = torch.full((2, 1, 1), 2.0 ** 119), torch.ones(2, 1, 1)
    q = torch.full((2, 1, 2, D), -100.0, dtype=torch.bfloat16)
    q[1] = 2.0 ** -120                                               # the second sequence's scores are ordinary ones
    for pages in (1, 200):
        bt = torch.full((2, pages), -1, dtype=torch.int32)
        bt[:, 0] = torch.tensor([0, 1])
        o, lse = ab.prefill_paged_q8(*to(cuda_device, q, kc, vc, ks, vs, bt, torch.tensor([1, 5], dtype=torch.int32)))
        assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
        assert (o[1] == 1).all() and torch.isfinite(lse[1]).all()
