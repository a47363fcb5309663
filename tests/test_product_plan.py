"""How the library splits a product over K, as the workspace it asks for tells: no GPU."""
import pytest

pytest.importorskip("torch")

from sparse_activation_ffn_amd import binding as pb  # noqa: E402


@pytest.mark.parametrize("m", [17, 29, 32])
def test_no_split_of_k_is_empty(m):
    """K is dealt out in pieces of 512, as many to every split: the last one has some.  (Of these m no smaller one asks for
    more: the workspace is that of this product, a float32 for each split and output.)"""
    split = 0
    for n in list(range(64, 4096, 56)) + [1000, 2752, 5120, 7168]:
        for k in (1024, 2080, 4096, 5120, 7168, 8192, 9216, 11008, 12288, 14336, 16384, 28672):
            need = pb.pi_mx_product_workspace_bytes(m, n, k)
            if need == 0:
                continue
            splits, pieces = need // (m * n * 4), -(-k // 512)
            assert splits > 1 and -(-splits * m * n * 4 // 256) * 256 == need
            each = -(-pieces // splits)
            assert (splits - 1) * each < pieces, (n, k, splits)
            split += 1
    assert split > 300
