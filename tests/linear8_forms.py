"""Sizes (m, n, k) of kaio_linear_w8a8 that run every kernel form there is, with k a multiple of 128 and not.

(One to five blocks of 128 k, so that rings are longer and shorter than the sum; tiles taken one after the other by one
workgroup for the forms that do so.  tests/test_linear8_forms_host.py holds the sizes against the selection itself.)
"""
SIZES = [
    # strips of 16 channels, 16 waves and 4; of 16-bit tokens rounded in the product's workgroups and before it
    (1, 1000, 384), (16, 1003, 528), (7, 4100, 2064), (16, 520, 4096), (8, 520, 4096), (8, 520, 4112), (3, 4001, 2064), (2, 8200, 400), (16, 8201, 1024),
    # 32 x 32, 32 x 64, 64 x 32, 64 x 64, 64 x 128 (channels x tokens): sets of waves
    (17, 200, 128), (40, 1000, 400), (61, 2048, 256), (96, 4096, 128), (120, 4001, 400), (512, 1024, 640), (24, 11004, 128),
    (32, 10000, 272), (61, 11004, 256), (250, 4096, 400), (1000, 1000, 1008), (128, 11004, 128), (384, 4001, 400),
    # 128 x 128, 128 x 256, 256 x 256: one tile for each workgroup, and several
    (256, 11004, 128), (700, 4096, 272), (1024, 4096, 640), (100, 40000, 272), (100, 40000, 256), (512, 11004, 144), (2048, 4001, 256),
    (2304, 8200, 128), (2304, 8200, 400), (1024, 16000, 384), (4096, 4096, 128), (4001, 4003, 528), (6000, 5000, 128),
    (6000, 5001, 400),
]
