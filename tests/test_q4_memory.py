"""What the structs of the rotary append and of the 4-bit cache hold of their tensors, without a GPU."""
import gc
import weakref

import pytest
import torch

from block_sparse_long_resa_b200 import resa as R
from block_sparse_long_resa_b200.cache import LayerCache, LayerCacheQ4


def test_structs_keep_their_lengths_and_tables():
    """A struct holds addresses: the lengths made for one call live as long as it does."""
    table = torch.zeros(2, 3, dtype=torch.int32)
    c4 = LayerCacheQ4.empty(6, 2, 16, 64, table)
    k = torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16)
    c16 = LayerCache(k, k, c4.desc, table, c4.seq_len)
    for make in (c4.struct, c4.select_struct, c16.struct):
        lens, rows = torch.tensor([5, 7], dtype=torch.int32), torch.tensor([1], dtype=torch.int32)
        seen = [weakref.ref(lens), weakref.ref(rows)]
        s = make(seq_len=lens, rows=rows)
        del lens, rows
        gc.collect()
        assert all(x() is not None for x in seen)
        assert s.seq_len == seen[0]().data_ptr() and s.rows == seen[1]().data_ptr()
        del s
        gc.collect()
        assert all(x() is None for x in seen)
    # and every other tensor that a 4-bit struct is made of
    args = [t.clone() for t in (c4.k, c4.k_sf, c4.v, c4.v_sf, c4.desc, table, c4.seq_len)]
    seen = [weakref.ref(t) for t in args]
    s = R.make_cache_q4(*args)
    del args
    gc.collect()
    assert all(x() is not None for x in seen)


def test_tokens_of_unlike_heads_are_refused():
    """k and v of other head counts, or heads of other sizes, would be read past their ends."""
    x = lambda h, d: torch.zeros(2, 5, h, d, dtype=torch.bfloat16)
    R.make_tokens(x(8, 64), x(2, 64), x(2, 64))
    for q, k, v in ((None, x(2, 64), x(1, 64)), (None, x(2, 64), x(4, 64)), (None, x(2, 128), x(2, 64)),
                    (None, x(2, 64), x(2, 128)), (x(8, 128), x(2, 64), x(2, 64)),
                    (x(8, 64), x(2, 128), x(2, 128))):
        with pytest.raises(R.ResaError) as e:
            R.make_tokens(q, k, v)
        assert e.value.status == 2
