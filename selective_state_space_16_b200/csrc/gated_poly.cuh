// generated by gen_gated_poly.py -- do not edit by hand
#pragma once
// max relative error of the fp32 evaluation 4.10e-08
#define SSM_GATED_DECAY_POLY {-0.4999999403953552f, 0.12499731779098511f, -0.020801063627004623f, 0.0024498903658241034f}
// max relative error of the fp32 evaluation 6.35e-08
#define SSM_GATED_WEIGHT_POLY {-0.24999761581420898f, 0.05202553793787956f, -0.0074114566668868065f}
// max relative error of the fp32 evaluation 6.14e-08
#define SSM_GATED_WEIGHT_INV_POLY {0.24999980628490448f, 0.010421709157526493f, -0.002642229199409485f}
