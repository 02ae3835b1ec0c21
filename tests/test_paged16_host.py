"""Refusals of the 16-bit paged cache's entry points (no GPU): every bad argument is answered before
anything is enqueued, and the binding refuses tensors it cannot hand on."""
import numpy as np
import pytest
import torch

from oracle import paged16

FAKE = 1 << 20  # a 16-byte-aligned non-null address; validation answers before any use

INVALID, UNSUPPORTED, WORKSPACE, CUDA = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from exact_tiled_attention_20_gb300 import _lib, build

    build.build_library()
    return _lib._load_paged16()


APPEND = dict(q=FAKE, k_new=FAKE, v_new=FAKE, q_stride=1024, k_stride=1024, v_stride=1024, q_out=FAKE, cu=None, table=FAKE,
              lens=FAKE, pos=None, cos=FAKE, sin=FAKE, k=FAKE, v=FAKE, B=2, total=4, Hq=8, Hkv=8, D=128, rot=128,
              inter=0, max_pos=100, num_pages=9, page=16, max_pages=4, dtype=0, stream=None)
TREE = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, mask=FAKE, o=FAKE, lse=None, B=2, Sq=4, Hq=16, Hkv=8, D=128,
            num_pages=9, page=16, max_pages=4, scale=0.1, ws=FAKE, ws_bytes=1 << 30, dtype=0, stream=None)
WINDOW = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, o=FAKE, lse=None, B=2, Sq=4, Hq=16, Hkv=8, D=128,
              num_pages=9, page=16, max_pages=4, scale=0.1, left=100, sinks=4, ws=FAKE, ws_bytes=1 << 30, dtype=0,
              stream=None)

POOL = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
        (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 4), INVALID), (dict(table=FAKE + 2), INVALID),
        (dict(lens=FAKE + 2), INVALID), (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(num_pages=0), INVALID),
        (dict(page=0), INVALID), (dict(page=-16), INVALID), (dict(max_pages=0), INVALID), (dict(D=80), UNSUPPORTED),
        (dict(D=0), UNSUPPORTED), (dict(D=512), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(B=1026), UNSUPPORTED),
        (dict(page=1 << 20, max_pages=1 << 11), UNSUPPORTED), (dict(page=16, max_pages=(1 << 27) - 1), UNSUPPORTED)]
DECODE = POOL + [
    (dict(q=None), INVALID), (dict(q=FAKE + 2), INVALID), (dict(o=None), INVALID), (dict(o=FAKE + 8), INVALID),
    (dict(lse=FAKE + 2), INVALID), (dict(Sq=0), INVALID), (dict(Hq=0), INVALID), (dict(Hq=12), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-0.1), INVALID), (dict(page=24), UNSUPPORTED),
    (dict(page=1), UNSUPPORTED), (dict(Sq=257), UNSUPPORTED), (dict(Hq=8 * 129), UNSUPPORTED),
    (dict(num_pages=0x7fffffff), UNSUPPORTED), (dict(page=1 << 28, max_pages=1, Hkv=16, Hq=16, D=128), UNSUPPORTED),
    (dict(B=1024, Sq=256, Hq=1 << 13, Hkv=1 << 13), UNSUPPORTED)]


@pytest.mark.parametrize("change,code", POOL + [
    (dict(cu=FAKE + 1), INVALID), (dict(pos=FAKE + 2), INVALID), (dict(total=-2), INVALID), (dict(total=5), INVALID),
    (dict(Hq=-8), INVALID), (dict(k_new=None), INVALID), (dict(v_new=FAKE + 2), INVALID), (dict(q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(q_out=FAKE + 4), INVALID),
    (dict(k_stride=1016), INVALID), (dict(v_stride=1028), INVALID), (dict(q_stride=1000), INVALID),
    (dict(k_stride=-1024), INVALID), (dict(rot=-16), INVALID), (dict(rot=8), INVALID), (dict(rot=144), INVALID),
    (dict(cos=None), INVALID), (dict(sin=FAKE + 4), INVALID), (dict(max_pos=0), INVALID),
    (dict(page=(1 << 28) + 1, max_pages=1), UNSUPPORTED), (dict(total=1 << 28), UNSUPPORTED), (dict(total=0), 0),
    (dict(total=0, q=None, k_new=None, v_new=None, q_out=None), 0)])
def test_append_refuses(lib, change, code):
    assert lib.fa_kv_append_paged_rope(*{**APPEND, **change}.values()) == code


@pytest.mark.parametrize("change,code", DECODE + [(dict(mask=None), INVALID), (dict(mask=FAKE + 2), INVALID)])
def test_tree_refuses(lib, change, code):
    assert lib.fa_decode_splitkv_paged_tree(*{**TREE, **change}.values()) == code


@pytest.mark.parametrize("change,code", DECODE + [(dict(left=-2), INVALID), (dict(sinks=-1), INVALID)])
def test_window_refuses(lib, change, code):
    assert lib.fa_decode_splitkv_paged_window(*{**WINDOW, **change}.values()) == code


@pytest.mark.parametrize("change", [dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=16)])
def test_decodes_refuse_a_bad_workspace(lib, change):
    want = WORKSPACE if torch.cuda.is_available() else CUDA  # without a device the SM count is not known
    assert lib.fa_decode_splitkv_paged_tree(*{**TREE, **change}.values()) == want
    assert lib.fa_decode_splitkv_paged_window(*{**WINDOW, **change}.values()) == want


def test_valid_calls_without_a_device_fail_loudly(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert lib.fa_kv_append_paged_rope(*APPEND.values()) == CUDA
    assert lib.fa_decode_splitkv_paged_tree(*TREE.values()) == CUDA
    assert lib.fa_decode_splitkv_paged_window(*WINDOW.values()) == CUDA


def test_workspace_bytes(lib):
    f = lib.fa_decode_paged_workspace_bytes
    rows = 2 * 152 * 12
    assert f(8, 3, 32, 8, 128, 152) == (rows * 512 + 255) // 256 * 256 + (rows * 4 + 255) // 256 * 256 + 16
    assert f(8, 64, 64, 8, 64, 152) == 2 * 152 * 256 * 65 * 4 + 16      # 512 query rows: row blocks of 256
    for bad in ((0, 1, 8, 8, 64), (1, 0, 8, 8, 64), (1, 1, 0, 8, 64), (1, 1, 9, 8, 64), (1, 1, 8, 8, 0)):
        assert f(*bad, 152) == 0


def test_binding_refuses_what_it_cannot_hand_on():
    import exact_tiled_attention_20_gb300 as fa

    x = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q, mask = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), torch.ones(1, 1, 1, dtype=torch.int32)
    with pytest.raises(TypeError):
        fa.fa_decode_splitkv_paged_window(q, x, x, table, lens)
    with pytest.raises(TypeError):
        fa.fa_decode_splitkv_paged_tree(q, x, x, table, lens, mask)
    with pytest.raises(TypeError):
        fa.fa_decode_splitkv_paged_tree(q, x, x, table, lens, None)
    with pytest.raises(TypeError):
        fa.fa_kv_append_paged_rope(q, q, x, x, table, lens)
    with pytest.raises(TypeError):
        fa.fa_kv_append_paged_rope(q, q, None, x, table, lens)
    with pytest.raises(ValueError):
        fa.fa_decode_splitkv_paged_window(q, x[0], x[0], table, lens)


def test_masks_of_the_reference():
    """The reference's masks against their definitions, said once more key by key."""
    rng = np.random.default_rng(0)
    for n, Sq in ((1, 1), (5, 3), (3, 5), (40, 33)):
        tree = paged16.random_trees(rng, 1, Sq)[0]
        words = paged16.pack_tree(tree).view(np.uint32)
        got, win = paged16.sees_tree(n, Sq, tree), paged16.sees_window(n, Sq, 4, 2)
        for i in range(Sq):
            assert tree[i, i] and not tree[i, i + 1:].any()
            for j in range(n):
                t = j - (n - Sq)
                assert got[i, j] == (t < 0 or bool(int(words[i, t // 32]) >> (t % 32) & 1))
                p = n - Sq + i
                assert win[i, j] == (j <= p and (j >= p - 4 or j < 2))
