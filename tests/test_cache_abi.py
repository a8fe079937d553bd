"""CPU tests of the paged cache's boundary: structs, masks, null contexts."""
import os
import re

import numpy as np
import pytest

from copy_reduce_dst_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tb():
    _build.build()
    from copy_reduce_dst_gb300 import tb as mod
    return mod


@pytest.mark.parametrize("name,cls", [("tb_kv_cache", "KvCacheStruct"), ("tb_tree", "Tree")])
def test_structs_match_header(tb, name, cls):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "tb.h")).read(), flags=re.S)
    end = text.index("} " + name + ";")
    body = text[text.rindex("typedef struct {", 0, end) + len("typedef struct {"):end]
    fields = []
    for line in body.split(";"):
        line = line.strip()
        if line:
            fields += [re.findall(r"\w+", part)[-1] for part in line.split(",")]
    assert fields == [n for n, _ in getattr(tb, cls)._fields_]


def test_limits_match_header(tb):
    text = open(os.path.join(ROOT, "include", "tb.h")).read()
    for name in ("TB_DTYPE_F16", "TB_DTYPE_BF16", "TB_DTYPE_F32", "TB_DTYPE_BYTE", "TB_KV_MAX_SLOTS",
                 "TB_TREE_MAX_SEQS"):
        assert int(re.search(rf"#define {name}\s+(\d+)", text).group(1)) == getattr(tb, name)


def test_null_context_is_rejected(tb):
    assert tb.lib.tb_kv_copy_pages(None, None, None, None, None, 0, None) == tb.TB_EINVAL
    assert tb.lib.tb_kv_resize(None, None, None, None, None) == tb.TB_EINVAL
    assert tb.lib.tb_kv_fork(None, None, None, None, None, None, None, None) == tb.TB_EINVAL
    assert tb.lib.tb_kv_compact(None, None, None, None, 0, None, None, None) == tb.TB_EINVAL
    assert tb.lib.tb_tree_attention(None, None, None) == tb.TB_EINVAL
    assert tb.lib.tb_tree_attention_workspace(None, None, 1, None) == tb.TB_EINVAL


def test_tree_mask(tb):
    assert tb.tree_mask([]) == []
    assert tb.tree_mask([-1, 0, 0, 1, -1]) == [[1], [3], [5], [11], [16]]
    chain = tb.tree_mask([i - 1 for i in range(70)])
    assert len(chain[0]) == 3 and chain[31] == [-1, 0, 0] and chain[69] == [-1, -1, 63]
    assert np.array(chain, np.int32).shape == (70, 3)
    with pytest.raises(ValueError):
        tb.tree_mask([-1, 1])


def test_descriptions_are_checked(tb):
    import torch
    pool = torch.zeros(1, 2, 4, 2, 8, dtype=torch.float16)
    with pytest.raises(ValueError):
        tb.kv_cache(pool, pool)  # on the host
    with pytest.raises(ValueError):
        tb.kv_cache(pool, None)
    with pytest.raises(ValueError):
        tb.kv_cache(layout="DHN")
