"""What include/qsa_chunk.h says about the size of the workspaces, held against the
size query (no GPU)."""
import re

import pytest

from test_chunk_host import _attend, lib  # noqa: F401
from test_header_bounds import _words


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tokens,hq,reqs", [
    (1, 2, 1), (12, 4, 4), (1000, 32, 4), (30000, 32, 12), (30000, 32, 3000), (2000000, 254, 65535),
    (16777216, 2, 65535), (5000, 510, 1), (65535, 2, 65535)])
def test_sizes_are_within_what_the_header_says(lib, dim, tokens, hq, reqs):  # noqa: F811
    words = _words("qsa_chunk.h", "qsa_chunk_attention_workspace_bytes")
    pieces, each = re.search(r"head_dim \* ([\d.]+) MB at most .* and (\d+) bytes for each token and "
                             r"request besides", words).groups()
    element, row = re.search(r"twice that and (\d+) bytes for each element of q, (\d+) for each of "
                             r"its rows and heads", words).groups()
    view = dict(dim=dim, ks0=32 * dim, ks1=2 * dim, ks2=dim, vs0=32 * dim, vs1=2 * dim, vs2=dim)
    chunk, prefix = (_attend(lib, x, True, tokens=tokens, hq=hq, reqs=reqs, **view)
                     for x in (False, True))
    fixed = int(float(pieces) * 1e6 * dim) + int(each) * (tokens + reqs)
    grows = (int(element) * dim + int(row)) * tokens * hq
    assert 0 < chunk <= fixed
    assert grows < prefix <= 2 * fixed + grows


def test_the_size_that_the_header_quotes(lib):  # noqa: F811
    view = dict(dim=128, ks0=4096, ks1=256, ks2=128, vs0=4096, vs1=256, vs2=128)
    need = _attend(lib, True, True, tokens=30000, hq=32, reqs=12, **view)
    assert "30000 tokens of 32 heads of 128: 1 GB" in _words("qsa_chunk.h", "qsa_chunk_attention_workspace_bytes")
    assert 0.95e9 < need < 1.1e9
