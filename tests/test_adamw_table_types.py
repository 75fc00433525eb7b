"""An AdamW table says which types its arrays have, so that a launch of other types does not follow it: the bytes of
the table, on the CPU."""
import ctypes
import itertools

import routing_grouped_expert_fp32_amd as bm
from test_abi import A

F32, BF, E4 = bm.BEAM_F32, bm.BEAM_BF16, bm.BEAM_FP8_E4M3


def _head(p, g, s, copy, counts=(1000, 0)):
    t = (bm._AdamWTensor * len(counts))()
    for i, n in enumerate(counts):
        for j, k in enumerate(("param", "grad", "m", "v", "m_scale", "v_scale", "copy")):
            if not (k.endswith("scale") and s == F32 or k == "copy" and not copy):
                setattr(t[i], k, A[0] + (8 * i + j) * (1 << 16))
        t[i].count = n
    size = bm.lib().beam_moe_adamw_table_bytes(t, len(counts))
    host = (ctypes.c_char * size)()
    assert bm.lib().beam_moe_adamw_table(t, len(counts), p, g, s, host, size) == 0
    return bytes(host[:16])


def test_tables_of_other_types_differ_in_their_heads():
    kinds = [k for k in itertools.product((F32, BF), (F32, BF), (F32, E4), (False, True)) if not (k[0] == BF and k[3])]
    heads = [_head(*k) for k in kinds]
    assert len(set(heads)) == len(kinds) == 12
    # the tensors without values say nothing, nor does their number's order
    assert all(_head(*k, counts=(0, 1000)) == h for k, h in zip(kinds, heads))
    assert bytes(16) not in heads
