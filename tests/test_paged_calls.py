"""What the Python calls hand to the library, and which tensors they take (no GPU: nothing is launched)."""
import ctypes

import torch

from gated_deltanet_linear_09_gb300 import build as gbuild
from gated_deltanet_linear_09_gb300 import gdn, runtime


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_tables_carry_their_width():
    """A row of a table has its own number of entries, whatever the distance of the rows."""
    def batch(table):
        return runtime.KVBatch(ints(table.shape[0] + 1), ints(table.shape[0]), table, 4).c
    for table, ld, cols in ((ints(3, 5), 5, 5), (ints(3, 8)[:, 2:4], 8, 2), (ints(1, 6).expand(3, 6), 0, 6),
                            (ints(1, 8)[:, :3], 3, 3), (ints(3, 0), 0, 0)):
        b = batch(table)
        assert (b.table_ld, b.table_cols) == (ld, cols)
    assert gdn.gdn_kv_batch.table_cols.offset == gdn.gdn_kv_batch.max_tokens.offset + 4


def test_table_width_is_checked():
    gbuild.build()
    A = 0x10000
    cache = gdn.gdn_kv_cache(A, A, None, None, 4, 16, 2, 128, gdn.GDN_KV_BF16, None)

    def read(**kw):
        d = dict(cu_seqlens=A, kv_lens=A, block_table=A, num_seqs=1, total_tokens=1, table_ld=4, max_tokens=1)
        return gdn.load().gdn_kv_read(ctypes.byref(cache), ctypes.byref(gdn.gdn_kv_batch(**{**d, **kw})), A + 2, A, None)
    assert read(table_cols=-1) == -1
    assert read(table_ld=0, table_cols=3, block_table=None) == -1
    assert read(table_ld=0, table_cols=3) == -7                     # (on to the next check: k is misaligned)
