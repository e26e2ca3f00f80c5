"""Sizes that reach each form of the dense layer with bias on a GPU of 148 SMs, and
the library's own answer to which form takes a size."""
import ctypes

TOKENS, TILES, PAIRS = 0, 1, 2
SMS = 148

# (kind, columns of a tile, parts of K), of the few-row kernel (kind, features of a block,
# warps): sizes M, K, N. None of them fills a tile: the
# last rows' tile holds one row, a few, or most of its rows (pairs: with and without
# rows for its odd half), parts of K and shares of rows are uneven, and the persistent
# pairs' third size gives each more than two tiles.
FORMS = {
    (TOKENS, 8, 8): [(1, 216, 72), (8, 1032, 2376), (16, 200, 3544), (11, 4040, 1000)],
    (TOKENS, 8, 16): [(1, 4104, 72), (8, 8968, 1544), (5, 4096, 2368)],
    (TOKENS, 16, 8): [(1, 200, 4744), (8, 4104, 4760), (16, 264, 7096), (9, 4088, 3560)],
    (TILES, 64, 1): [(129, 216, 72), (17, 208, 72), (188, 216, 72)],
    (TILES, 64, 2): [(137, 904, 1416), (17, 912, 2936), (199, 912, 1416)],
    (TILES, 64, 3): [(129, 696, 712), (18, 664, 1416), (189, 656, 720)],
    (TILES, 64, 4): [(129, 784, 456), (17, 792, 1096), (189, 808, 456)],
    (TILES, 64, 5): [(129, 528, 72), (18, 520, 72), (189, 528, 72)],
    (TILES, 64, 6): [(129, 656, 80), (18, 648, 88), (188, 656, 72)],
    (TILES, 64, 7): [(133, 784, 72), (17, 784, 80), (188, 776, 72)],
    (TILES, 64, 8): [(131, 912, 72), (17, 912, 72), (188, 944, 72)],
    (TILES, 128, 1): [(138, 200, 4808), (9, 200, 9576), (189, 208, 4744)],
    (TILES, 128, 2): [(131, 3544, 3032), (9, 4328, 5872), (197, 3480, 2896)],
    (TILES, 128, 3): [(144, 2464, 2416), (17, 2696, 4744), (194, 2448, 2376)],
    (TILES, 128, 4): [(136, 4888, 1680), (9, 5128, 3464), (194, 4912, 1704)],
    (TILES, 128, 5): [(133, 3680, 1448), (11, 4120, 2904), (195, 3600, 1432)],
    (TILES, 128, 6): [(134, 7384, 1056), (9, 7672, 2136), (188, 7304, 1032)],
    (TILES, 128, 8): [(131, 9776, 856), (9, 9792, 1808), (188, 9904, 840)],
    (PAIRS, 192, 1): [(398, 200, 4760), (259, 200, 6608), (840, 200, 7856)],
    (PAIRS, 192, 2): [(395, 2952, 2968), (513, 3136, 1912), (200, 2952, 5672)],
    (PAIRS, 192, 3): [(398, 3400, 1424), (258, 3672, 2032), (190, 3368, 2960)],
    (PAIRS, 192, 4): [(644, 2912, 920), (571, 6544, 928), (193, 2952, 2832)],
    (PAIRS, 256, 1): [(410, 264, 7200), (258, 264, 7352), (1400, 200, 9416)],
    (PAIRS, 256, 2): [(398, 4280, 3096), (279, 4304, 3176), (328, 4256, 3280)],
    (PAIRS, 256, 3): [(401, 2832, 2432), (2317, 2888, 464), (191, 2904, 4792)],
    (PAIRS, 256, 4): [(400, 5064, 1488), (524, 5032, 1160), (189, 5040, 2904)],
}

# Sizes whose loop over K is long, for waits that run out; K * 2^-10 is exact in bf16.
LONG = {
    (TILES, 64, 1): (24, 1536, 8960),
    (TILES, 64, 5): (24, 4096, 1536),
    (TILES, 128, 1): (129, 1536, 8960),
    (TILES, 128, 2): (24, 4096, 8960),
    (TILES, 128, 8): (800, 10240, 256),
    (PAIRS, 192, 1): (600, 1536, 4096),
    (PAIRS, 192, 2): (600, 4096, 2048),
    (PAIRS, 192, 3): (129, 4096, 4096),
    (PAIRS, 256, 1): (300, 1536, 8960),
    (PAIRS, 256, 2): (300, 5120, 4096),
    (PAIRS, 256, 4): (400, 5120, 1536),
}


class _Form(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("cols", ctypes.c_int32), ("parts", ctypes.c_int32)]


def form_of(lib, M, K, N, sms=SMS):
    f = _Form()
    lib.wavei_dense_form(ctypes.c_int32(sms), ctypes.c_int32(M), ctypes.c_int32(K), ctypes.c_int32(N),
                         ctypes.byref(f))
    return f.kind, f.cols, f.parts


def name(form):
    return f"{('tokens', 'tiles', 'pairs')[form[0]]}-{form[1]}-{form[2]}"
