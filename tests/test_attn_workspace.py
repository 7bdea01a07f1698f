"""What cache_attention_workspace_size asks for, and which sizes it takes (host
alone): partial sums are those that the kernels can leave, not one for every
tile that there might be.

Few query rows: a wave leaves at most two tiles' sums, and there are no more waves
than the chip holds (8 a CU with heads of 128, 16 of 64, 4 of 256); a tile's are
its rows, of head_dim + 2 values each; and 8 bytes name the waves of each tile.  Many: tiles of 128 rows are
cut into ranges of tokens only while there are no more than 512 of those."""
import pytest

WAVES = {64: 4096, 128: 2048, 256: 1024}


def size(t, d, hq, hkv, window=0, sinks=0, page=64, **kw):
    q = dict(n_seqs=1, rows=1, max_rows=1, max_context=30000, max_pages=1024)
    q.update(kw)
    return t.cache_attention_workspace_size(
        dict(n_pages=8, page_tokens=page, n_kv_heads=hkv, head_dim=d), q, hq, window, sinks)


def few_rows(d, tile, units):
    return 2 * WAVES[d] * tile * (d + 2) * 4 + 8 * units + 256


@pytest.mark.parametrize("rows", [100, 8192, 32768, 200000])
def test_prompts_of_heads_of_256(tsl_lib, rows):
    for hq, hkv in ((64, 8), (8, 8), (7, 1)):
        units = hkv * -(-rows * (hq // hkv) // 16)
        assert 0 < size(tsl_lib, 256, hq, hkv, rows=rows, max_rows=rows) <= few_rows(256, 16, units)


@pytest.mark.parametrize("d,hq,hkv", [(64, 32, 8), (128, 64, 8), (256, 64, 8), (128, 28, 4)])
@pytest.mark.parametrize("n", [1, 33, 1000])
def test_generated_tokens(tsl_lib, d, hq, hkv, n):
    for rows in (1, 2, 5):
        per = rows * hq // hkv
        assert size(tsl_lib, d, hq, hkv, n_seqs=n, rows=n * rows, max_rows=rows) <= \
            few_rows(d, 16, n * hkv * -(-per // 4))


def test_one_long_prompt_of_heads_of_256_beside_many_tokens(tsl_lib):
    """600 sequences, 8 query heads a K/V head, the longest with 1024 rows: accepted,
    whatever 600 of the longest would come to."""
    kw = dict(n_seqs=600, rows=1623, max_rows=1024, max_pages=32)
    assert 0 < size(tsl_lib, 256, 32, 4, **kw) <= few_rows(256, 16, 600 * 4 * 512)
    # tiles of the kernel of few rows without partial sums: four a workgroup
    size(tsl_lib, 128, 64, 16, n_seqs=65535, rows=70000, max_rows=1024)


@pytest.mark.parametrize("n,rows", [(256, 9), (1024, 9), (16000, 9), (2048, 128), (60000, 33), (65535, 64)])
def test_many_sequences_of_many_rows(tsl_lib, n, rows):
    """Up to the stated limits, and no more partial sums than can be; with three
    tiles or more, 1 GiB of expanded records beside them."""
    for d, hq, hkv in ((128, 64, 8), (64, 32, 8), (128, 28, 4)):
        images = (1 << 30) + (1 << 21) if rows * hq // hkv > 256 else 0
        most = 512 * 128 * (d + 2) * 4 + few_rows(d, 16, n * hkv * 16) + images
        assert size(tsl_lib, d, hq, hkv, n_seqs=n, rows=min(n * rows, (1 << 22) - 1), max_rows=rows) <= most


def test_records_are_counted_in_32_bits(tsl_lib):
    """A call is divided by its records only where their number, rounded up to a
    multiple of the waves, stays below 2^31: 1023 tiles of 2099202 records do not."""
    assert size(tsl_lib, 128, 1, 1, page=32, n_seqs=1023, rows=1023, max_pages=2099202) == 0
    assert size(tsl_lib, 128, 1, 1, page=32, n_seqs=1023, rows=1023, max_pages=2099202 - 5) > 0
