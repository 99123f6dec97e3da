"""The sizes of the GPU tests reach every tile of the shared expert's bf16 products, whole and in k-splits."""
import shared_tiles
import test_gpu_block


def test_every_tile_is_reached():
    want = {(p, t, split) for p in ("gate and up", "down", "dh") for t in range(5) for split in (False, True)}
    want |= {("gradients", t, split) for t in range(3) for split in (False, True)}
    got = {(p, t, s > 1) for size in test_gpu_block.TILE_SIZES for p, (t, s) in shared_tiles.tiles(*size).items()}
    assert got == want, want - got


def test_the_rule_stays_in_its_limits():
    """Splits keep four k-tiles each, and a launch's sums stay under what the workspace holds."""
    for T in (33, 65, 300, 777, 2049, 16384):
        for d, f in ((64, 64), (2048, 1408), (333, 517), (7168, 2048), (40, 11000), (5000, 24)):
            for p, (t, s) in shared_tiles.tiles(T, d, f).items():
                k = {"gate and up": d, "down": f, "dh": d}.get(p, max(2 * f, T))
                assert 0 <= t < (3 if p == "gradients" else 5) and (s == 1 or s <= 16 and -(-(k + 7) // 64) // s >= 4), (T, d, f, p)
