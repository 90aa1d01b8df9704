"""What a user reads about the operators of shared pages, and their host-side arithmetic (no GPU)."""

def test_the_documentation_says_when_to_compact():
    from decode_serving_gb300.paged import PagedCache
    for f in (PagedCache.fork, PagedCache.compact):
        assert "between steps, when every token is" in " ".join(f.__doc__.split()).lower()
