"""The 8-bit decode where the two warpgroups of a CTA hand O over to one another: sequences of
two to four tiles, one after another in the same CTA, so that the hand-over's buffer is written for one
part as soon as the part before has read it."""

import numpy as np
import pytest
import torch

import attention_online_softmax_fwd_b200 as ab
from attention_online_softmax_fwd_b200 import inputs as gen
from oracle import attn_oracle as orc
from parity_util import compare_output

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 128), (8, 2, 128), (16, 2, 128), (32, 2, 128), (12, 6, 64), (16, 2, 64),
                                      (32, 2, 64)])
def test_hand_over_of_many_short_parts(cuda_device, kind, Hq, Hkv, D):
    """Tolerances: those of parity_util. The calls repeat bit for bit."""
    g = torch.Generator().manual_seed(7000 + Hq + Hkv + D)
    rows = 900
    lens = torch.tensor([130, 257, 385, 512, 129, 256, 300], dtype=torch.int32)
    cache = gen.paged_decode_inputs(7, Hq, Hkv, D, 32, 0, 0, seed=7001 + Hq, lens=lens.tolist(), max_pages=16,
                                    poison=False)
    kc, ks = gen.quantize_pool_q8(cache.k_pages, 16, kind)
    vc, vs = gen.quantize_pool_q8(cache.v_pages, 16, kind)
    which = torch.randint(0, 7, (rows,), generator=g)          # every sequence many times, in any order
    scale = gen.attn_scale(D)
    o_ref, l_ref = orc.decode_paged_q8(cache.q, kc, vc, ks, vs, cache.block_table, cache.seq_lens, scale)
    pick = which.numpy()
    args = [t.to(cuda_device) for t in (cache.q[which], kc, vc, ks, vs, cache.block_table[which], lens[which])]
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    o, lse = ab.decode_paged_q8(*args, scale=scale, device_status=st)
    compare_output(o, o_ref[pick], lse, l_ref[pick], label=f"{kind} {Hq}/{Hkv}x{D}")
    for _ in range(5):
        o2, l2 = ab.decode_paged_q8(*args, scale=scale, device_status=st)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert int(st) == 0
    # a row's result does not depend on where in the batch it stands
    for i in range(7):
        same = o[which.to(cuda_device) == i]
        assert torch.equal(same, same[:1].expand_as(same))
    assert np.isfinite(lse.cpu().numpy()).all()
