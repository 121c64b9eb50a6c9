"""Sizes (T, D, F) at which the rule of csrc/dense_pick.cu takes each kernel, whatever number of
clusters the device holds at once: tests/test_dense_pick_host.py holds the rule to them,
tests/test_gpu_dense_kernels.py runs them.  A kernel is (kind, tile columns, K splits)."""

FORWARD = {
    ("few", 0, 0): [(1, 72, 136), (17, 1000, 264), (32, 520, 200)],
    ("pair", 128, 1): [(70, 136, 200), (5000, 520, 264)],
    ("pair", 128, 2): [(777, 1544, 776), (300, 1544, 1544)],
    ("pair", 128, 4): [(70, 1032, 72), (130, 1544, 200)],
    ("pair", 256, 1): [(777, 520, 2824), (9000, 264, 2824), (9000, 1032, 1368)],
    ("pair", 256, 2): [(267, 6336, 2752), (351, 5632, 2912)],
    ("pair", 256, 4): [(341, 7096, 1160), (83, 7336, 2544)],
}
GATED = {
    ("few", 0, 0): [(1, 72, 136), (33, 1000, 72), (64, 520, 200)],
    ("pair", 256, 1): [(70, 136, 200), (3000, 264, 1368)],
    ("pair", 256, 2): [(777, 1544, 776), (300, 1544, 1544)],
    ("pair", 256, 4): [(70, 1032, 72), (130, 1544, 200)],
}
INPUT_GRADIENT = {
    ("pair", 128, 1): [(70, 136, 200), (5000, 264, 520)],
    ("pair", 128, 2): [(777, 776, 1544)],
    ("pair", 128, 4): [(70, 72, 1032), (130, 200, 1544)],
    ("pair", 256, 1): [(777, 2824, 520), (9000, 2824, 264)],
    ("pair", 256, 2): [(267, 2752, 6336)],
    ("pair", 256, 4): [(341, 1160, 7096), (83, 2544, 7336)],
}
WEIGHT_GRADIENT = {
    ("pair", 128, 1): [(70, 136, 200), (200, 1032, 776)],
    ("pair", 128, 2): [(1477, 2840, 88), (1450, 2640, 120)],
    ("pair", 128, 4): [(1030, 72, 136), (3001, 264, 200)],
    ("pair", 256, 1): [(520, 1032, 2824), (520, 2824, 4104)],
    ("pair", 256, 2): [(6448, 960, 1136), (5967, 680, 1560)],
    ("pair", 256, 4): [(8192, 1184, 272), (9034, 152, 2448)],
}
# both at once: one launch (kind "grads", of its tile columns), or the two kernels picked alone
BOTH_GRADIENTS = {
    ("grads", 128): [(70, 136, 200), (1030, 520, 520)],
    ("grads", 256): [(2050, 1032, 4104), (9000, 520, 2824)],
    ("pair", "pair"): [(33000, 776, 776)],
}
FORMS = {"forward": (0, False, FORWARD), "gated": (0, True, GATED), "input": (1, False, INPUT_GRADIENT),
         "weight": (2, False, WEIGHT_GRADIENT)}
# clusters of 2, 4 and 8 CTAs that run at once: 76 pairs on 152 SMs; the larger ones fit fewer SMs
CLUSTERS = [(76, b, c) for b in (28, 32, 36, 38) for c in (10, 12, 15, 17, 19)]
