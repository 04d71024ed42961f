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
